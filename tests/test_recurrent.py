"""The rule token by token over a pool of states (kda_recurrent, kda_gdn_recurrent)
against the recurrence in fp64."""
import ctypes

import numpy as np
import pytest

from ops_ref import within

P = ctypes.c_void_p(0x10000)   # never dereferenced


def steps(S, q, k, v, g, beta):
    """S [H, K, V], the others [T, H, ...]: yields (o, S) after each token."""
    for t in range(q.shape[0]):
        S = np.exp(g[t])[..., None] * S
        e = v[t] - np.einsum("hk,hkv->hv", k[t], S)
        S = S + np.einsum("hk,hv->hkv", k[t], beta[t][:, None] * e)
        yield np.einsum("hk,hkv->hv", q[t], S), S


# ------------------------------------------------------------------------- CPU

def test_reference_against_oracle():
    import oracle
    import workloads as W
    inp = W.make_inputs(W.variant("tiny_fp32", T=6, H=2, h0=True), 1)
    x = [u[0].astype(np.float64) for u in (inp.q, inp.k, inp.v, inp.g, inp.beta)]
    got = list(steps(inp.h0[0].astype(np.float64), *x))
    o, hT = oracle.kda_ref_fwd(inp.q, inp.k, inp.v, inp.g, inp.beta, h0=inp.h0)
    assert np.allclose([y for y, _ in got], o[0], rtol=1e-12, atol=1e-12)
    assert np.allclose(got[-1][1], hT[0], rtol=1e-12, atol=1e-12)


def test_refusals():
    import gated_delta_rule_63_amd as kda
    L = kda.lib()

    def call(fn, B=2, T=3, H=2, K=128, N=None, dt=0, num=4, pdt=1, **kw):
        a = dict(zip("q k v g beta cu slots outs pool".split(), [P] * 9))
        a.update({"cu": None, **{x: y for x, y in kw.items() if x in a}})
        d = kda.Desc(B, T, H, K, 128, B if N is None else N, dt, 1, None, 0)
        return getattr(L, fn)(*a.values(), num, pdt, kw.get("o", P), ctypes.byref(d), None)

    M = ctypes.c_void_p(0x10004)
    for fn in ("kda_recurrent", "kda_gdn_recurrent"):
        for name in ("q", "k", "v", "g", "beta", "pool", "o"):
            assert call(fn, **{name: None}) == -1, name
        for name in ("q", "k", "v", "pool", "o", "g"):
            assert call(fn, **{name: M}) == -3, name               # not 16-byte aligned
        assert call(fn, K=64) == -3 and call(fn, dt=5) == -4 and call(fn, pdt=2) == -4
        assert call(fn, N=3) == -2 and call(fn, num=-1) == -2
        assert call(fn, slots=None, num=1) == -2                   # fewer slots than sequences
        assert call(fn, B=1 << 20, H=16) == -2                     # 2^24 chains
        assert call(fn, T=0, pool=None) == 0                       # nothing to do
        assert call(fn, num=0, pool=None) == 0 and call(fn, num=0, q=None) == -1   # a pool without slots


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    from gated_delta_rule_63_amd import _ops
    q, g, b = torch.zeros(2, 3, 4, 128), torch.zeros(2, 3, 4, 128), torch.zeros(2, 3, 4)
    pool, i = torch.zeros(5, 4, 128, 128), lambda *s: torch.zeros(*s, dtype=torch.int32)
    chk = lambda pool=pool, slots=i(2), outs=i(2, 3), cu=None, out=None, g=g, s=False: _ops._check_recurrent(
        q, q, q, g, b, pool, slots, outs, cu, out, s, _device=False)
    chk()
    chk(g=b, s=True)
    chk(pool=pool.bfloat16(), slots=None, outs=None, out=torch.zeros(2, 3, 4, 128))
    for kw in (dict(pool=pool[:, :3]), dict(pool=pool.half()), dict(pool=pool[:1], slots=None), dict(slots=i(3)),
               dict(slots=torch.zeros(2, dtype=torch.int64)), dict(outs=i(2, 4)), dict(out=torch.zeros(2, 3, 4, 64)),
               dict(pool=pool.transpose(2, 3)), dict(g=b), dict(cu=i(3))):
        with pytest.raises(ValueError):
            chk(**kw)


# ------------------------------------------------------------------------- GPU

@pytest.fixture
def torch_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def make(torch, B, T, H, dtype, scalar, P, pool_dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    x = dict(q=unit(n(B, T, H, 128)).to(dtype), k=unit(n(B, T, H, 128)).to(dtype), v=n(B, T, H, 128).to(dtype),
             g=-torch.nn.functional.softplus(n(B, T, H) if scalar else n(B, T, H, 128)), beta=torch.rand(B, T, H, generator=gen))
    return x, (0.1 * n(P, H, 128, 128)).to(pool_dtype), gen


CASES = [  # lengths (None: rows of T), T, B, H, inputs, gate, pool, out_slots
    (None, 1, 1, 1, "float32", False, "float32", False),
    (None, 1, 7, 3, "bfloat16", False, "bfloat16", False),
    (None, 1, 33, 9, "float32", True, "bfloat16", False),
    (None, 4, 40, 7, "bfloat16", False, "float32", True),
    (None, 17, 2, 5, "bfloat16", True, "float32", True),
    ((0, 3, 1, 0, 70, 5), 79, 6, 2, "float32", False, "float32", False),
    ((1, 0, 8, 2), 11, 4, 3, "bfloat16", False, "bfloat16", True),
    # above 1.5 (sequence, head) pairs a compute unit: four waves a head
    (None, 1, 45, 9, "float32", True, "bfloat16", False),
    (None, 4, 56, 7, "bfloat16", False, "float32", True),
    ((0, 3, 1, 0, 7, 5), 16, 6, 66, "bfloat16", True, "float32", False),
    ((2, 9, 0, 1), 12, 4, 97, "float32", False, "bfloat16", True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,T,N,H,dtype,scalar,pool_dtype,keep", CASES)
def test_recurrent(torch_gpu, lens, T, N, H, dtype, scalar, pool_dtype, keep):
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    rows, P = (1 if lens else N), 2 * N + N * T
    x, pool, gen = make(torch, rows, T, H, getattr(torch, dtype), scalar, P, getattr(torch, pool_dtype), 11)
    order = torch.randperm(P, generator=gen).to(torch.int32)
    slots = order[:N].clone()
    if N > 3:
        slots[1], slots[3] = -1, P + 5                     # empty places of the batch
    outs = order[N:N + rows * T].reshape(rows, T).clone() if keep else None
    if keep:
        outs[0, 0] = -1
        outs[-1, -1] = P
    cu = torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32) if lens else None
    dev = lambda t: None if t is None else t.cuda()
    d = {n: t.cuda() for n, t in x.items()}
    got_pool, out = pool.cuda(), torch.full((rows, T, H, 128), 3.0, device="cuda")
    f = kda.gdn_recurrent if scalar else kda.recurrent
    ret = f(d["q"], d["k"], d["v"], d["g"], d["beta"], got_pool, slots=dev(slots), out_slots=dev(outs), cu_seqlens=dev(cu),
            out=out)
    torch.cuda.synchronize()
    assert ret is out
    ref_o, ref_pool = np.full((rows, T, H, 128), 3.0), pool.double().numpy().copy()
    written = set()
    for n in range(N):
        s = int(slots[n])
        if not 0 <= s < P:
            continue
        row, t0, t1 = (0, int(cu[n]), int(cu[n + 1])) if lens else (n, 0, T)
        a = [x[u][row, t0:t1].double().numpy() for u in ("q", "k", "v", "g", "beta")]
        if scalar:
            a[3] = a[3][..., None]
        start = pool[s].double().numpy()
        for t, (o, S) in enumerate(steps(start, *a)):
            ref_o[row, t0 + t] = o
            to = int(outs[row, t0 + t]) if keep else (s if t0 + t + 1 == t1 else -1)
            if 0 <= to < P:
                ref_pool[to] = S
                written.add(to)
    within(out.cpu().numpy(), ref_o, "o")
    half = 2.0 ** -8 if pool_dtype == "bfloat16" else 0.0
    w = sorted(written)
    if w:
        within(got_pool[w].float().cpu().numpy(), ref_pool[w], "states", half)
    rest = [i for i in range(P) if i not in written]
    assert torch.equal(got_pool[rest].cpu(), pool[rest])       # bit for bit as they were
    for n in range(N):
        if not 0 <= int(slots[n]) < P:
            part = out[0, int(cu[n]):int(cu[n + 1])] if lens else out[n]
            assert bool((part == 3.0).all())


@pytest.mark.gpu
def test_far_slots(torch_gpu):
    """A slot whose elements lie beyond 2^31."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    x, pool, _ = make(torch, 1, 2, 1, torch.float32, False, 1, torch.bfloat16, 4)
    big = torch.empty(140001, 1, 128, 128, dtype=torch.bfloat16, device="cuda")
    big[140000], big[9] = pool[0].cuda(), 0.0
    d = {n: t.cuda() for n, t in x.items()}
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    o = kda.recurrent(d["q"], d["k"], d["v"], d["g"], d["beta"], big, slots=i(140000), out_slots=i(139999, 140000))
    small = pool.cuda().repeat(2, 1, 1, 1)
    want = kda.recurrent(d["q"], d["k"], d["v"], d["g"], d["beta"], small, slots=i(1), out_slots=i(0, 1))
    assert torch.equal(o, want) and torch.equal(big[139999:], small) and not bool(big[9].any())


@pytest.mark.gpu
def test_as_decode_step_in_a_graph(torch_gpu):
    """Steps captured into a graph and replayed are the decode step's, slot by slot."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    x, pool, _ = make(torch, 5, 1, 4, torch.bfloat16, False, 5, torch.float32, 6)
    d = {n: t.cuda() for n, t in x.items()}
    args = [d[n] for n in ("q", "k", "v", "g", "beta")]
    slots = torch.tensor([3, 0, 4, 1, 2], dtype=torch.int32, device="cuda")
    mine, out = pool.cuda(), torch.empty(5, 1, 4, 128, device="cuda")
    run = lambda: kda.recurrent(*args, mine, slots=slots, out=out)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    state = pool.cuda()[slots.long()].contiguous()
    kda.decode_step(*args, state=state, in_place=True)
    for rep in range(3):
        graph.replay()
        o, _ = kda.decode_step(*args, state=state, in_place=True)
        torch.cuda.synchronize()
        within(out.cpu().numpy(), o.cpu().numpy(), f"replay {rep} o")
        within(mine[slots.long()].cpu().numpy(), state.cpu().numpy(), f"replay {rep} state")


@pytest.mark.gpu
def test_draft_and_accept(torch_gpu):
    """Serving as it is done: a prefill, four drafted tokens with every state kept,
    two of them accepted, and on from there; against the recurrence over the accepted
    tokens. fp32 inputs: the prefill is accurate to 1e-4 of the state's RMS."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    x, _, _ = make(torch, 1, 60, 3, torch.float32, False, 1, torch.float32, 8)
    d = {n: t.cuda() for n, t in x.items()}
    part = lambda a, b: [d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")]
    pool = torch.zeros(6, 3, 128, 128, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kda.fwd(*part(0, 50), final_state=pool[2:3])
    kda.recurrent(*part(50, 54), pool, slots=i(2), out_slots=i(0, 1, 3, 4))
    o = kda.recurrent(*part(52, 60), pool, slots=i(1))          # on from the second draft's state
    ref = list(steps(np.zeros((3, 128, 128)), *(x[n][0].double().numpy() for n in ("q", "k", "v", "g", "beta"))))
    within(o[0].cpu().numpy(), np.stack([y for y, _ in ref[52:]]), "o", tol=2e-4)
    within(pool[1].cpu().numpy(), ref[-1][1], "state", tol=2e-4)


@pytest.mark.gpu
def test_scalar_gate_of_a_slice(torch_gpu):
    """A slice of tokens whose gates do not start on 16 bytes is refused, before anything
    runs, and its clone is taken."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    x, pool, _ = make(torch, 1, 6, 3, torch.float32, True, 1, torch.float32, 9)
    part = [x[n].cuda()[:, 1:4] for n in ("q", "k", "v", "g", "beta")]
    p, start = pool.cuda(), pool.cuda()
    assert part[3].is_contiguous() and part[3].data_ptr() % 16
    with pytest.raises(kda.KDAError) as e:
        kda.gdn_recurrent(*part, p)
    assert e.value.code == -3 and torch.equal(p, start)
    part[3] = part[3].clone()
    o = kda.gdn_recurrent(*part, p)
    a = [x[n][0, 1:4].double().numpy() for n in ("q", "k", "v", "g", "beta")]
    a[3] = a[3][..., None]
    ref = list(steps(pool[0].double().numpy(), *a))
    within(o[0].cpu().numpy(), np.stack([y for y, _ in ref]), "o")
    within(p[0].cpu().numpy(), ref[-1][1], "state")


@pytest.mark.gpu
@pytest.mark.parametrize("pool_dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,H,scalar", [(2, 3, False), (3, 2, True), (70, 6, False), (39, 10, True)])
def test_bits_of_the_states(torch_gpu, pool_dtype, N, H, scalar):
    """The states' bits are those of fp32 arithmetic on the CPU, one rounding an
    operation, in the kernel's order: P^T k in eight sums over rows r, r + 8, ..., of
    which 0, 2, 4, 6 are added in turn, then 1, 3, 5, 7, then both. (The decays come from
    the kernel: e^g is what a state of ones becomes where k and beta are zero.) Eight
    waves a head and four, 6 and 420 or 390 pairs on 256 compute units."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    T = 3
    x, pool, _ = make(torch, N, T, H, torch.bfloat16, scalar, N, getattr(torch, pool_dtype), 23)
    d = {n: t.cuda() for n, t in x.items()}
    f = kda.gdn_recurrent if scalar else kda.recurrent
    ones = torch.ones(N * T, H, 128, 128, device="cuda")
    zero, flat = torch.zeros(N * T, 1, H, 128, device="cuda"), lambda t: t.reshape(N * T, 1, *t.shape[2:])
    f(zero, zero, zero, flat(d["g"]), torch.zeros(N * T, 1, H, device="cuda"), ones)
    decay = ones[..., :1].reshape(N, T, H, 128, 1).cpu().numpy()
    got = pool.cuda()
    f(*(d[n] for n in ("q", "k", "v", "g", "beta")), got)
    S = pool.float().numpy()
    k, v, beta = (x[n].float().numpy() for n in ("k", "v", "beta"))
    for t in range(T):
        Pt = S * decay[:, t]
        kk = k[:, t, :, :, None]
        pk = (Pt * kk).reshape(N, H, 16, 8, 128)
        a = pk[:, :, 0]
        for m in range(1, 16):
            a = a + pk[:, :, m]
        half = [((a[:, :, i] + a[:, :, i + 2]) + a[:, :, i + 4]) + a[:, :, i + 6] for i in (0, 1)]
        be = beta[:, t, :, None] * (v[:, t] - (half[0] + half[1]))
        S = Pt + kk * be[:, :, None, :]
        assert S.dtype == np.float32
    assert torch.equal(got.cpu(), torch.from_numpy(S).to(got.dtype))

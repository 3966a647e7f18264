"""The rule with a vector state (kda_scan, its gradient, and token by token over a pool)
against the recurrence in fp64."""
import ctypes

import numpy as np
import pytest

import layers_ref as R

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(0x10000)   # never dereferenced


# ------------------------------------------------------------------------- CPU

@pytest.mark.parametrize("leaky", [False, True])
def test_reference_gradient_against_differences(leaky):
    """The adjoint against central differences of the recurrence, in fp64."""
    rng = np.random.default_rng(1)
    bounds = R.bounds_of((4, 0, 3), 1, 7)
    x, g, dy = rng.normal(size=(1, 7, 2)), -rng.random((1, 7, 2)), rng.normal(size=(1, 7, 2))
    h0, dhT = rng.normal(size=(3, 2)), rng.normal(size=(3, 2))

    def loss(x, g, h0):
        h, hT, _, _ = R.scan(x, g, bounds, h0, leaky)
        return float((h * dy).sum() + (hT * dhT).sum())

    got, _ = R.scan_bwd(x, g, dy, bounds, h0, dhT, leaky)
    for k, (v, d) in enumerate(zip((x, g, h0), got)):
        for at in np.ndindex(v.shape):
            args = [u.copy() for u in (x, g, h0)]
            args[k][at] += 1e-5
            up = loss(*args)
            args[k][at] -= 2e-5
            assert abs((up - loss(*args)) / 2e-5 - d[at]) < 1e-8


def test_refusals():
    import gated_delta_rule_63_amd as kda
    L = kda.lib()
    D = lambda B=2, T=3, C=5, N=None, dt=0, ws=None, n=0: kda._lib.ScanDesc(B, T, C, B if N is None else N, dt, 0, ws, n)
    call = lambda d=None, x=P, g=P, cu=None, y=P: L.kda_scan(x, g, cu, P, y, P, P, d if d is None else ctypes.byref(d), None)
    assert call(None) == -1
    for kw in ("x", "g", "y"):
        assert call(D(), **{kw: None}) == -1, kw
    for d in (D(B=0), D(T=-1), D(C=0), D(N=3), D(N=-1, B=1), D(T=(1 << 30) + 1), D(C=(1 << 20) + 1),
              D(B=1 << 17, C=1 << 13), D(B=1 << 16, T=1 << 20, C=64)):
        assert call(d) == -2, (d.B, d.T, d.C, d.num_seqs)
    assert call(D(), cu=P) == -2 and call(D(B=1, N=4)) == -2        # packed needs one row; N rows without cu
    assert call(D(dt=2)) == -4
    assert call(D(B=1, T=0, N=0), x=None, g=None, y=None, cu=P) == 0    # no sequence: nothing to do
    bwd = lambda d, states=P, dy=P, dx=P, dg=P: L.kda_scan_bwd(P, P, None, P, states, dy, P, dx, dg, P, ctypes.byref(d), None)
    for kw in ("dy", "dx", "dg"):
        assert bwd(D(), **{kw: None}) == -1
    need = L.kda_scan_bwd_workspace_size(ctypes.byref(D()), 0)
    assert need >= 2 * 5 * 4 and bwd(D(), states=None) == -5 and bwd(D(ws=P, n=need - 1), states=None) == -5
    assert bwd(D(ws=ctypes.c_void_p(0x10004), n=need), states=None) == -3
    for f in (L.kda_scan_workspace_size, lambda d: L.kda_scan_bwd_workspace_size(d, 0), lambda d: L.kda_scan_states_rows(d, 0)):
        assert f(None) == 0 and f(ctypes.byref(D(C=0))) == 0
    rows = lambda d, packed: L.kda_scan_states_rows(ctypes.byref(d), packed)
    assert rows(D(T=129), 0) == 4 and rows(D(B=1, T=129, N=7), 1) == 8 and rows(D(), 1) == 0 and rows(D(B=1, N=7), 0) == 0
    rec = lambda d, num=4, pdt=1, slots=P, pool=P, y=P: L.kda_scan_recurrent(P, P, None, slots, P, pool, num, pdt, y, ctypes.byref(d), None)
    assert rec(D(), pool=None) == -1 and rec(D(), y=None) == -1 and rec(D(), pdt=2) == -4 and rec(D(), num=-1) == -2
    assert rec(D(), slots=None, num=1) == -2 and rec(D(T=0), pool=None) == 0 and rec(D(), num=0, pool=None) == 0


def test_binding_refusals():
    from gated_delta_rule_63_amd import _layers as M
    z = torch.zeros
    x, g, i = z(2, 3, 4, 5), z(2, 3, 4, 5), lambda *s: z(*s, dtype=torch.int32)
    h, st = z(2, 4, 5), z(2, 1, 4, 5)
    chk = lambda x=x, g=g, dy=x, cu=None, h0=h, dhT=h, states=st: M._check_scan_bwd(x, g, dy, cu, h0, dhT, states, _device=False)
    chk()
    chk(h0=None, dhT=None, states=None)
    y = z(1, 3, 20, dtype=torch.bfloat16)
    chk(x=y, g=z(1, 3, 20), dy=y, cu=i(3), h0=z(2, 20), dhT=z(2, 20), states=z(1, 2, 20))
    for kw in (dict(x=x.half()), dict(x=z(2, 3)), dict(g=g.bfloat16()), dict(g=z(2, 3, 20)), dict(dy=x.bfloat16()), dict(cu=i(3)),
               dict(h0=z(3, 4, 5)), dict(dhT=z(2, 20)), dict(states=z(2, 2, 4, 5)), dict(g=z(2, 3, 5, 4).transpose(2, 3)),
               dict(h0=h.bfloat16())):
        with pytest.raises(ValueError):
            chk(**kw)
    with pytest.raises(ValueError):
        M._check_scan(x, g, None)                       # not on a GPU
    pool = z(5, 4, 5)
    rec = lambda pool=pool, slots=i(2), outs=i(2, 3), out=None: M._check_scan_recurrent(x, g, pool, slots, outs, None, out, _device=False)
    rec()
    rec(pool=pool.bfloat16(), slots=None, outs=None, out=x.clone())
    for kw in (dict(pool=z(5, 20)), dict(pool=pool.half()), dict(pool=pool[:1], slots=None), dict(slots=i(3)), dict(outs=i(2, 4)),
               dict(slots=z(2, dtype=torch.int64)), dict(out=x.bfloat16()), dict(pool=z(5, 5, 4).transpose(1, 2))):
        with pytest.raises(ValueError):
            rec(**kw)


def test_sizes_beyond_32_bits():
    """2^32 + 3 of anything is refused, not taken for 3. (Tensors without storage: only shapes are looked at.)"""
    from gated_delta_rule_63_amd import _layers as M
    n = (1 << 32) + 3
    e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="meta")
    for shape in ((1, n, 1), (n, 1, 1), (1, 1, n), (1, 1, 1 << 20, 1 << 13)):
        with pytest.raises(ValueError, match="32 bits"):
            M._check_scan(e(*shape), e(*shape), None, _device=False)
        with pytest.raises(ValueError, match="32 bits"):
            M.scan_workspace_size(e(*shape))
    with pytest.raises(ValueError, match="32 bits"):
        M._check_scan(e(1, 3, 1), e(1, 3, 1), e(n, dtype=torch.int32), _device=False)
    with pytest.raises(ValueError, match="32 bits"):
        M._check_scan_recurrent(e(2, 1, 1), e(2, 1, 1), e(n, 1), e(2, dtype=torch.int32), None, None, None, _device=False)


# ------------------------------------------------------------------------- GPU

@pytest.fixture
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_63_amd as kda
    return kda


def make(B, T, C, dtype, lens, state, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    N = B if lens is None else len(lens)
    rate = torch.exp(torch.rand(C, generator=gen) * 6.2 - 6.2)           # memories of 1 to 500 tokens
    return dict(x=n(B, T, C).to(getattr(torch, dtype)), g=-2 * rate * torch.sigmoid(n(B, T, C)), dy=n(B, T, C).to(getattr(torch, dtype)),
                h0=n(N, C) if state else None, dhT=n(N, C) if state else None,
                cu=torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32) if lens else None)


def on(t):
    return None if t is None else t.cuda()


def as64(t):
    return None if t is None else t.double().cpu().numpy()


def kept_at(states, bounds, packed, n, j):
    r, t0, _ = bounds[n]
    return states[0, t0 // 128 + n + j] if packed else states[r, j]


CASES = [  # lengths (None: rows of T), B, T, C, type, leaky, states both ways
    (None, 1, 1, 1, "float32", False, False),
    (None, 3, 1, 65, "bfloat16", True, True),
    (None, 1, 15, 64, "float32", True, True),
    (None, 2, 16, 63, "bfloat16", False, False),
    (None, 2, 17, 130, "float32", False, True),
    (None, 1, 127, 3, "bfloat16", True, False),
    (None, 2, 128, 64, "float32", False, False),
    (None, 1, 129, 200, "bfloat16", False, True),
    (None, 1, 256, 64, "float32", True, True),
    (None, 2, 257, 100, "bfloat16", False, True),
    (None, 3, 1001, 70, "float32", False, True),
    (None, 1, 2100, 33, "bfloat16", True, True),
    ((0, 3, 0, 128, 1, 257, 0), 1, 389, 65, "float32", False, True),
    ((130, 5, 300, 0, 64), 1, 499, 64, "bfloat16", True, True),
    ((1, 2, 3, 127, 129, 700), 1, 962, 5, "float32", True, False),
    # the other forms: 64 and 32 channels a workgroup, and a sequence's chunks side by side
    (None, 40, 150, 260, "bfloat16", False, True),
    (None, 40, 300, 130, "float32", True, True),
    (None, 1, 9000, 40, "bfloat16", False, True),
    (None, 1, 4300, 67, "float32", True, False),
    ((3000, 0, 1, 2500, 129), 1, 5630, 34, "bfloat16", True, True),
    ((900, 0, 70, 1500, 129), 1, 2599, 1000, "float32", False, True),
    # with the chunks' fold in a launch of its own
    (None, 1, 33000, 20, "bfloat16", True, True),
    (None, 1, 12800, 1300, "float32", False, True),
    ((20000, 0, 13001), 1, 33001, 33, "float32", False, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,B,T,C,dtype,leaky,state", CASES)
def test_scan(kda, lens, B, T, C, dtype, leaky, state):
    s = make(B, T, C, dtype, lens, state, 3)
    y, hT, kept = kda.scan(on(s["x"]), on(s["g"]), cu_seqlens=on(s["cu"]), initial_state=on(s["h0"]), leaky=leaky,
                           output_chunk_states=True)
    torch.cuda.synchronize()
    bounds = R.bounds_of(lens, B, T)
    h, rT, e, eT = R.scan(as64(s["x"]), as64(s["g"]), bounds, as64(s["h0"]), leaky)
    R.held(as64(y), h, e, "y", dtype, 1e-5)
    R.held(as64(hT), rT, eT, "hT", rms=1e-5)
    for n, (r, t0, t1) in enumerate(bounds):
        for j, t in enumerate(range(t0, t1, 128)):
            start = np.zeros(C) if s["h0"] is None else as64(s["h0"])[n]
            R.held(as64(kept_at(kept, bounds, lens is not None, n, j)), start if t == t0 else h[r, t - 1],
                   0.0 if t == t0 else e[r, t - 1], f"state {n}, {j}")


@pytest.mark.gpu
@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("lens,B,T,C,dtype,leaky,state", CASES)
def test_scan_bwd(kda, lens, B, T, C, dtype, leaky, state, known):
    s = make(B, T, C, dtype, lens, state, 4)
    x, g, cu, h0 = on(s["x"]), on(s["g"]), on(s["cu"]), on(s["h0"])
    kept = kda.scan(x, g, cu_seqlens=cu, initial_state=h0, leaky=leaky, output_chunk_states=True)[2] if known else None
    got = kda.scan_bwd(x, g, on(s["dy"]), cu_seqlens=cu, initial_state=h0, d_final_state=on(s["dhT"]), chunk_states=kept,
                       leaky=leaky)
    torch.cuda.synchronize()
    ref, off = R.scan_bwd(as64(s["x"]), as64(s["g"]), as64(s["dy"]), R.bounds_of(lens, B, T), as64(s["h0"]), as64(s["dhT"]), leaky)
    for u, r, e, what, t in zip(got, ref, off, ("dx", "dg", "dh0"), (dtype, "float32", "float32")):
        R.held(as64(u), r, e, what, t, 1e-5)


@pytest.mark.gpu
def test_resets_ones_and_strong_gates(kda):
    """Gates of -inf (a reset), 0 (a running sum), -100 and -1e-9, mixed; forwards and back."""
    s = make(1, 300, 66, "float32", None, True, 5)
    gen = torch.Generator().manual_seed(6)
    choice = torch.tensor([-float("inf"), 0.0, -100.0, -1e-9, -0.5])
    s["g"] = choice[torch.randint(0, 5, s["g"].shape, generator=gen)]
    s["g"][:, :, :2] = 0.0
    s["g"][:, 150, 1] = -float("inf")
    for leaky in (False, True):
        y, hT, kept = kda.scan(on(s["x"]), on(s["g"]), initial_state=on(s["h0"]), leaky=leaky, output_chunk_states=True)
        d = kda.scan_bwd(on(s["x"]), on(s["g"]), on(s["dy"]), initial_state=on(s["h0"]), d_final_state=on(s["dhT"]),
                         chunk_states=kept, leaky=leaky)
        torch.cuda.synchronize()
        bounds = R.bounds_of(None, 1, 300)
        a = [as64(s[n]) for n in ("x", "g")]
        h, rT, e, eT = R.scan(*a, bounds, as64(s["h0"]), leaky)
        R.held(as64(y), h, e, "y")
        R.held(as64(hT), rT, eT, "hT")
        ref, off = R.scan_bwd(*a, as64(s["dy"]), bounds, as64(s["h0"]), as64(s["dhT"]), leaky)
        for u, r, b, what in zip(d, ref, off, ("dx", "dg", "dh0")):
            R.held(as64(u), r, b, what)


@pytest.mark.gpu
def test_rows_outside_the_sequences_and_in_place(kda):
    """Rows before the first and behind the last sequence stay as they were, and a call may
    write over its own x, or dy."""
    s = make(1, 400, 67, "bfloat16", None, False, 7)
    cu = torch.tensor([10, 140, 140, 333], dtype=torch.int32)
    bounds = [(0, 10, 140), (0, 140, 140), (0, 140, 333)]
    x, g, dy = on(s["x"]), on(s["g"]), on(s["dy"])
    y, hT, kept = kda.scan(x, g, cu_seqlens=cu.cuda(), output_chunk_states=True)
    again = x.clone()
    out, _, _ = kda.scan(again, g, cu_seqlens=cu.cuda(), out=again)
    inside = slice(10, 333)
    assert out is again and torch.equal(again[:, inside], y[:, inside])
    assert torch.equal(again[:, :10], x[:, :10]) and torch.equal(again[:, 333:], x[:, 333:])
    h, rT, e, eT = R.scan(as64(s["x"]), as64(s["g"]), bounds)
    R.held(as64(y[:, inside]), h[:, inside], e[:, inside], "y", "bfloat16")
    R.held(as64(hT), rT, eT, "hT")
    # through the C entry point: dx in dy's place, dg in a tensor of sevens
    d, dg, dh0 = dy.clone(), torch.full_like(g, 7.0), torch.empty(3, 67, device="cuda")
    desc = kda._lib.ScanDesc(1, 400, 67, 3, 0, 0, None, 0)
    need = kda.lib().kda_scan_bwd_workspace_size(ctypes.byref(desc), 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    desc.workspace, desc.workspace_bytes = ws.data_ptr() or None, need
    p, c = lambda t: ctypes.c_void_p(t.data_ptr()), cu.cuda()
    assert kda.lib().kda_scan_bwd(p(x), p(g), p(c), None, p(kept), p(d), None, p(d), p(dg), p(dh0), ctypes.byref(desc),
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    ref, off = R.scan_bwd(as64(s["x"]), as64(s["g"]), as64(s["dy"]), bounds)
    R.held(as64(d[:, inside]), ref[0][:, inside], off[0][:, inside], "dx", "bfloat16")
    R.held(as64(dg[:, inside]), ref[1][:, inside], off[1][:, inside], "dg")
    R.held(as64(dh0), ref[2], off[2], "dh0")
    for u, was in ((d, dy), (dg, torch.full_like(g, 7.0))):
        assert torch.equal(u[:, :10], was[:, :10]) and torch.equal(u[:, 333:], was[:, 333:])


@pytest.mark.gpu
@pytest.mark.parametrize("T,C", [(300, 40), (8000, 40), (9000, 40), (33000, 40), (150, 10400)])
def test_states_in_place(kda, T, C):
    """The last state written over the first one, and the gradients' alike, in each form."""
    s = make(1, T, C, "bfloat16", None, True, 13)
    x, g, dy, h0, dhT = (on(s[n]) for n in ("x", "g", "dy", "h0", "dhT"))
    y, hT, kept = kda.scan(x, g, initial_state=h0, output_chunk_states=True)
    h = h0.clone()
    y2, out, _ = kda.scan(x, g, initial_state=h, final_state=h)
    bound = 2 * 500 * 6 * R.U                      # (the folds may be grouped otherwise: two results within one bound)
    assert out is h and float((h - hT).abs().max()) <= bound * float(hT.abs().max())
    assert float((y2.float() - y.float()).abs().max()) <= (2.0 ** -7 + bound) * float(y.float().abs().max())
    desc = kda._lib.ScanDesc(1, T, C, 1, 0, 0, None, 0)
    need = kda.lib().kda_scan_bwd_workspace_size(ctypes.byref(desc), 1)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), need
    dx, dg, dh0 = kda.scan_bwd(x, g, dy, initial_state=h0, d_final_state=dhT, chunk_states=kept)
    d, dx2, dg2, p = dhT.clone(), torch.empty_like(dx), torch.empty_like(dg), lambda t: ctypes.c_void_p(t.data_ptr())
    assert kda.lib().kda_scan_bwd(p(x), p(g), None, p(h0), p(kept), p(dy), p(d), p(dx2), p(dg2), p(d), ctypes.byref(desc),
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert float((d - dh0).abs().max()) <= bound * float(dh0.abs().max())
    assert float((dg2 - dg).abs().max()) <= bound * float(dg.abs().max())
    assert float((dx2.float() - dx.float()).abs().max()) <= (2.0 ** -7 + bound) * float(dx.float().abs().max())


@pytest.mark.gpu
def test_empty_calls(kda):
    z = lambda *s: torch.zeros(*s, device="cuda")
    h0 = torch.ones(2, 5, device="cuda")
    y, hT, kept = kda.scan(z(2, 0, 5), z(2, 0, 5), initial_state=h0, output_chunk_states=True)
    assert y.shape == (2, 0, 5) and torch.equal(hT, h0) and kept.shape == (2, 0, 5)
    assert torch.equal(kda.scan(z(2, 0, 5), z(2, 0, 5))[1], z(2, 5))
    dx, dg, dh0 = kda.scan_bwd(z(2, 0, 5), z(2, 0, 5), z(2, 0, 5), d_final_state=h0)
    assert dx.shape == (2, 0, 5) and torch.equal(dh0, h0)


@pytest.mark.gpu
def test_beyond_32_bit_offsets(kda):
    """3.3e9 elements; the last tokens against a call that starts from the state before them."""
    T, C = 1 << 20, 3201
    x = torch.empty(1, T, C, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    g = torch.full((1, T, C), -0.05, device="cuda")
    cut = T - 300
    h = kda.scan(x[:, :cut], g[:, :cut])[1]
    want, wT, _ = kda.scan(x[:, cut:].clone(), g[:, cut:].clone(), initial_state=h)
    y, hT, kept = kda.scan(x, g, output_chunk_states=True)
    # the tiles lie otherwise, so roundings differ: two results of one bound, 20 tokens of memory
    assert float((hT - wT).abs().max()) <= 2 * 20 * 6 * R.U * float(hT.abs().max())
    assert float((y[:, cut:].float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.abs().max())
    del y, want
    dy = torch.ones_like(x)
    dx, dg, _ = kda.scan_bwd(x, g, dy, chunk_states=kept)
    sx, sg, _ = kda.scan_bwd(x[:, cut:].clone(), g[:, cut:].clone(), dy[:, cut:].clone(), initial_state=h)
    assert float((dx[:, cut:].float() - sx.float()).abs().max()) <= 2.0 ** -7 * float(sx.max())
    assert float((dg[:, cut:] - sg).abs().max()) <= 4 * 20 * 6 * R.U * float(sg.abs().max())


@pytest.mark.gpu
def test_four_gibibytes_of_a_sequence(kda):
    """Few channels over so many tokens that the rows left from a token on are 2^32 bytes and some.
    Decays of one between resets every 100 tokens, inputs of -1, 0 and 1: all sums are exact."""
    C, every = 64, 100
    T = (1 << 24) + 64
    cycle = torch.randint(-1, 2, (every, C), generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(T, C, device="cuda")
    g[::every] = float("-inf")
    want = torch.empty_like(x)
    ahead = torch.empty_like(x)                     # sums to the next reset: of dx with dy = x
    whole = T // every * every
    x[:whole].view(-1, every, C)[:] = cycle
    x[whole:] = cycle[:T - whole]
    want[:whole].view(-1, every, C)[:] = cycle.cumsum(0)
    want[whole:] = cycle.cumsum(0)[:T - whole]
    ahead[:whole].view(-1, every, C)[:] = cycle.flip(0).cumsum(0).flip(0)
    ahead[whole:] = cycle[:T - whole].flip(0).cumsum(0).flip(0)
    y, hT, kept = kda.scan(x[None], g[None], output_chunk_states=True)
    assert torch.equal(y[0], want) and torch.equal(hT[0], want[-1].float())
    assert torch.equal(kept[0, 1:], want[127::128][:kept.shape[1] - 1].float())
    for states in (kept, None):
        dx, dg, _ = kda.scan_bwd(x[None], g[None], x[None], chunk_states=states)
        assert torch.equal(dx[0], ahead)
        assert torch.equal(dg[0, 1:every], want[:every - 1].float() * ahead[1:every].float())
        assert torch.equal(dg[0, 1 - every - T % every:][:every - 1], dg[0, 1:every]) and not dg[0, ::every].any()
        del dx, dg


POOL = [  # lengths, T, N, C, inputs, pool, leaky, out_slots
    (None, 1, 1, 1, "float32", "float32", False, False),
    (None, 1, 70, 128, "bfloat16", "bfloat16", False, False),
    (None, 5, 9, 65, "float32", "bfloat16", True, True),
    (None, 17, 3, 64, "bfloat16", "float32", False, True),
    ((0, 3, 1, 0, 40, 5), 49, 6, 34, "float32", "float32", True, False),
    ((1, 0, 8, 2), 11, 4, 256, "bfloat16", "bfloat16", True, True),
    (None, 1, 300, 1000, "bfloat16", "float32", False, False),
    (None, 2, 7, 301, "bfloat16", "float32", True, False),
    (None, 1, 1027, 6, "float32", "bfloat16", False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,T,N,C,dtype,pool_dtype,leaky,keep", POOL)
def test_scan_recurrent(kda, lens, T, N, C, dtype, pool_dtype, leaky, keep):
    rows, slots_n = (1 if lens else N), 2 * N + N * T
    s = make(rows, T, C, dtype, lens, False, 8)
    gen = torch.Generator().manual_seed(9)
    pool = torch.randn(slots_n, C, generator=gen).to(getattr(torch, pool_dtype))
    order = torch.randperm(slots_n, generator=gen).to(torch.int32)
    slots = order[:N].clone()
    if N > 3:
        slots[1], slots[3] = -1, slots_n + 5
    outs = order[N:N + rows * T].reshape(rows, T).clone() if keep else None
    if keep:
        outs[0, 0], outs[-1, -1] = -1, slots_n
    got, out = pool.cuda(), torch.full((rows, T, C), 3.0, device="cuda", dtype=getattr(torch, dtype))
    assert kda.scan_recurrent(on(s["x"]), on(s["g"]), got, slots=on(slots), out_slots=on(outs), cu_seqlens=on(s["cu"]),
                              leaky=leaky, out=out) is out
    torch.cuda.synchronize()
    bounds = R.bounds_of(lens, rows, T)
    want, bound = pool.double().numpy(), np.zeros((slots_n, C))
    y, ey, written = np.full((rows, T, C), 3.0), np.zeros((rows, T, C)), set()
    for n, (r, t0, t1) in enumerate(bounds):
        at = int(slots[n])
        if not 0 <= at < slots_n:
            continue
        h, _, e, _ = R.scan(as64(s["x"])[r:r + 1], as64(s["g"])[r:r + 1], [(0, t0, t1)], pool[at].double().numpy()[None], leaky)
        y[r, t0:t1], ey[r, t0:t1] = h[0, t0:t1], e[0, t0:t1]
        for t in range(t0, t1):
            to = int(outs[r, t]) if keep else (at if t + 1 == t1 else -1)
            if 0 <= to < slots_n:
                want[to], bound[to] = h[0, t], e[0, t]
                written.add(to)
    R.held(as64(out), y, ey, "y", dtype)
    w = sorted(written)
    R.held(as64(got)[w], want[w], bound[w], "states", pool_dtype)
    rest = [i for i in range(slots_n) if i not in written]
    assert torch.equal(got[rest].cpu(), pool[rest])


@pytest.mark.gpu
def test_unaligned_tensors(kda):
    """Tensors that start on no 16 bytes give the same bits."""
    s = make(5, 3, 128, "bfloat16", None, False, 12)
    x, g, dy, pool = on(s["x"]), on(s["g"]), on(s["dy"]), torch.randn(5, 128, device="cuda")
    flat = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].reshape(t.shape)
    ux, ug, udy, up = flat(x), flat(g), flat(dy), flat(pool)
    assert ux.data_ptr() % 16 and up.data_ptr() % 16
    assert torch.equal(kda.scan_recurrent(x, g, pool), kda.scan_recurrent(ux, ug, up)) and torch.equal(pool, up)
    y, hT, kept = kda.scan(x, g, initial_state=pool, output_chunk_states=True)
    uy, uhT, ukept = kda.scan(ux, ug, initial_state=up, output_chunk_states=True)
    assert torch.equal(y, uy) and torch.equal(hT, uhT) and torch.equal(kept, ukept)
    for a, b in zip(kda.scan_bwd(x, g, dy, initial_state=pool, d_final_state=hT), kda.scan_bwd(ux, ug, udy, initial_state=up, d_final_state=flat(hT))):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_prompt_then_tokens(kda):
    """A prompt by scan() into a slot of the pool, then token by token, against the whole."""
    s = make(1, 150, 4 * 32, "float32", None, False, 10)
    x, g = on(s["x"]).reshape(1, 150, 4, 32), on(s["g"]).reshape(1, 150, 4, 32)
    pool = torch.zeros(3, 4, 32, device="cuda")
    kda.scan(x[:, :140].contiguous(), g[:, :140].contiguous(), final_state=pool[2:3])
    slot = torch.tensor([2], dtype=torch.int32, device="cuda")
    ys = [kda.scan_recurrent(x[:, t:t + 1].contiguous(), g[:, t:t + 1].contiguous(), pool, slots=slot) for t in range(140, 150)]
    torch.cuda.synchronize()
    h, hT, e, eT = R.scan(as64(s["x"]), as64(s["g"]), R.bounds_of(None, 1, 150))
    R.held(as64(torch.cat(ys, 1)).reshape(1, 10, 128), h[:, 140:], e[:, 140:], "y")
    R.held(as64(pool[2]).reshape(1, 128), hT, eT, "state")
    assert not bool(pool[:2].any())


@pytest.mark.gpu
def test_streams_and_graphs(kda):
    """The same bits on another stream, in two calls at once, and in a replayed graph, with
    work between the replays; the gradient with its workspace alike."""
    s = make(2, 700, 192, "bfloat16", None, True, 11)
    x, g, dy, h0, dhT = (on(s[n]) for n in ("x", "g", "dy", "h0", "dhT"))
    both = lambda stream=None: (*kda.scan(x, g, initial_state=h0, output_chunk_states=True, stream=stream),
                                *kda.scan_bwd(x, g, dy, initial_state=h0, d_final_state=dhT, stream=stream))
    want = both()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [both(st) for st in sides]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        for u in held:
            u.fill_(1.0)
        graph.replay()
        other = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)) and all(torch.equal(a, b) for a, b in zip(other, want))


def growing(B, T, C, dtype, lens, leaky, seed):
    """Gates above zero, in nine kinds of channels whose states, and gradients, stay finite
    throughout: growth over zeros (slow, fast and within a few tokens) until inputs come, a tiny state that grows, growth
    and decay in turn, a reset after growth, a large state that decays and grows back, ordinary
    decays, and differences of bounded values."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    u = lambda *s: torch.rand(*s, generator=gen)
    bounds = R.bounds_of(lens, B, T)
    x, dy, g = n(B, T, C), n(B, T, C), torch.zeros(B, T, C)
    h0, dhT = torch.zeros(len(bounds), C), torch.zeros(len(bounds), C)
    for s, (r, t0, t1) in enumerate(bounds):
        k, at, half = t1 - t0, slice(t0, t1), (t1 - t0) // 2
        if k == 0:
            continue
        for kind, gate, window in ((0, 0.05, 400), (1, 0.7, 60), (8, 12.0, 4)):
            g[r, at, kind::9] = gate
            x[r, t0:max(t1 - window, t0), kind::9] = 0.0
            dy[r, min(t0 + window, t1):t1, kind::9] = 0.0
        g[r, at, 2::9] = min(5.0, 100.0 / k)
        x[r, at, 2::9] = dy[r, at, 2::9] = 0.0
        h0[s, 2::9] = dhT[s, 2::9] = 1e-30
        g[r, at, 3::9] = (60.0 - 120.0 * (torch.arange(k) % 2))[:, None]
        g[r, at, 4::9] = 0.7
        g[r, t0 + half:t1, 4::9] = -0.5
        g[r, t0 + half, 4::9] = -float("inf")
        x[r, t0:t0 + half, 4::9] = 0.0
        dy[r, min(t0 + 60, t0 + half):t0 + half, 4::9] = 0.0
        if half:
            step = min(80.0, 40.0 * half) / half
            g[r, t0:t0 + half, 5::9] = -step
            g[r, t0 + half:t0 + 2 * half, 5::9] = step
        x[r, at, 5::9] = dy[r, at, 5::9] = 0.0
        h0[s, 5::9], dhT[s, 5::9] = 1e20, 1e-10
        g[r, at, 6::9] = -2 * u(k, C)[:, 6::9]
        w = 20 * u(k + 1, C)[:, 7::9] - 10
        g[r, at, 7::9] = w[1:] - w[:-1]
    dt = getattr(torch, dtype)
    return dict(x=x.to(dt), g=g, dy=dy.to(dt), h0=h0, dhT=dhT, bounds=bounds,
                cu=torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32) if lens else None)


GROWING = [  # lengths (None: rows of T), B, T, C, type
    (None, 2, 1, 16, "float32"),
    (None, 1, 128, 64, "float32"),                      # a workgroup a strip: 16, 32 and 64 channels
    (None, 2, 257, 100, "bfloat16"),
    (None, 40, 150, 260, "float32"),
    (None, 40, 300, 130, "bfloat16"),
    ((130, 5, 300, 0, 64), 1, 499, 64, "float32"),
    (None, 1, 4300, 67, "bfloat16"),                    # chunks side by side, each folding those before it
    (None, 1, 9000, 40, "float32"),
    ((900, 0, 70, 1500, 129), 1, 2599, 1000, "float32"),
    (None, 1, 33000, 24, "bfloat16"),                   # with the fold in a launch of its own
    (None, 1, 12800, 1300, "float32"),
    ((20000, 0, 13001), 1, 33001, 33, "float32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("leaky", [False, True])
@pytest.mark.parametrize("lens,B,T,C,dtype", GROWING)
def test_growing_gates(kda, lens, B, T, C, dtype, leaky):
    """Where no state overflows none of the composed decays does, in any form, forwards and back."""
    s = growing(B, T, C, dtype, lens, leaky, 14)
    x, g, dy, cu, h0, dhT = (on(s[n]) for n in ("x", "g", "dy", "cu", "h0", "dhT"))
    y, hT, kept = kda.scan(x, g, cu_seqlens=cu, initial_state=h0, leaky=leaky, output_chunk_states=True)
    grads = [kda.scan_bwd(x, g, dy, cu_seqlens=cu, initial_state=h0, d_final_state=dhT, chunk_states=states, leaky=leaky)
             for states in (kept, None)]
    torch.cuda.synchronize()
    args = [as64(s[n]) for n in ("x", "g")]
    back = lambda leaky: R.scan_bwd(*args, as64(s["dy"]), s["bounds"], as64(s["h0"]), as64(s["dhT"]), leaky)
    h, rT, e, eT = R.scan(*args, s["bounds"], as64(s["h0"]), leaky)
    ref, off = back(leaky)
    if leaky:
        # the factor 1 - e^g of an input is off by 2 e^g / (e^g - 1) + 1 half steps, 6.1 at most (g = 1/2), and its product
        # by one more: 8 where the references have 6. dx is off by |1 - e^g| times D's error (D is dx without the
        # factor), and by 8 half steps of its own
        (D, _, _), (eD, _, _) = back(False)
        f = np.abs(np.expm1(args[1]))
        off = (f * (eD - 5 * R.U * np.abs(D)) + 8 * R.U * f * np.abs(D), off[1] * 8 / 6, off[2])
        e, eT = e * 8 / 6, eT * 8 / 6
    R.held(as64(y), h, e, "y", dtype)
    R.held(as64(hT), rT, eT, "hT")
    for got, states in zip(grads, ("kept", "formed again")):
        for v, want, bound, what, t in zip(got, ref, off, ("dx", "dg", "dh0"), (dtype, "float32", "float32")):
            R.held(as64(v), want, bound, f"{what}, states {states}", t)

"""The residual's addition with an RMS norm (kda_add_norm), its 8-bit output and its
gradient, against the formulas in fp64."""
import ctypes

import numpy as np
import pytest

import layers_ref as R

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(0x10000)   # never dereferenced
EPS = 1e-5


def rel(C):
    """What fp32 leaves of y, relative: half of the sum of squares' C / 64 additions on a lane and
    at most 10 between lanes, two half steps each for the square, the division, the root
    and the reciprocal, one for each product."""
    return (0.5 * (C / 64 + 10 + 2) + 8) * R.U


def stream(x, res):
    """r as it is stored, and in fp64."""
    r = x if res is None else (x.float() + res.float()).to(res.dtype)
    return r, r.double().numpy()


def norm(r, w):
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + EPS) * w


def grad(r, w, dy, dr):
    """d, dw and their bounds."""
    C = r.shape[-1]
    k = 1.0 / np.sqrt((r * r).mean(-1, keepdims=True) + EPS)
    n, dn = r * k, dy * w
    d = k * (dn - n * (n * dn).mean(-1, keepdims=True)) + dr
    size = k * (np.abs(dn) + np.abs(n) * np.abs(n * dn).mean(-1, keepdims=True))
    # twice rel(C) for n and k, and as much again for the mean's sum; one addition for dr
    bd = size * (4 * rel(C) + 4 * R.U) + 2 * R.U * (np.abs(dr) + np.abs(d))
    dw = (dy * n).sum(0)
    return d, dw, bd, np.abs(dy * n).sum(0) * (rel(C) + (r.shape[0] + 20) * R.U)


def as64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------- CPU

def test_reference_gradient_against_differences():
    rng = np.random.default_rng(1)
    r, w, dy, dr = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    d, dw, _, _ = grad(r, w, dy, dr)
    loss = lambda r, w: float((norm(r, w) * dy + r * dr).sum())
    for v, want, put in ((r, d, lambda v: (v, w)), (w, dw, lambda v: (r, v))):
        for at in np.ndindex(v.shape):
            u = v.copy()
            u[at] += 1e-5
            up = loss(*put(u))
            u[at] -= 2e-5
            assert abs((up - loss(*put(u))) / 2e-5 - want[at]) < 1e-8


def test_refusals():
    import gated_delta_rule_63_amd as kda
    L = kda.lib()
    D = lambda rows=3, C=256, dt=0, res=0, ws=None, n=0: kda._lib.NormDesc(rows, C, dt, res, ws, n)
    ref = lambda d: None if d is None else ctypes.byref(d)
    M = ctypes.c_void_p(0x10004)
    fwd = lambda d, x=P, res=P, w=P, eps=EPS, y=P, r=P: L.kda_add_norm(x, res, w, eps, y, r, ref(d), None)
    q8 = lambda d, x=P, res=P, w=P, eps=EPS, group=128, q=P, s=P, r=P: L.kda_add_norm_q8(x, res, w, eps, group, q, s, r, ref(d), None)
    bwd = lambda d, r=P, w=P, eps=EPS, dy=P, dr=P, dx=P, dres=P, dw=P: L.kda_add_norm_bwd(r, w, eps, dy, dr, dx, dres, dw, ref(d), None)
    need = L.kda_add_norm_bwd_workspace_size(ref(D()))
    assert need > 0
    B = lambda **kw: D(ws=P, n=need, **kw)
    for f, d, names in ((fwd, D, ("x", "w", "y", "r")), (q8, D, ("x", "w", "q", "s", "r")), (bwd, B, ("r", "w", "dy", "dx", "dw"))):
        assert f(None) == -1
        for name in names:
            assert f(d(), **{name: None}) == -1, name
        for bad in (d(rows=-1), d(rows=1 << 31), d(C=0), d(C=16385)):
            assert f(bad) == -2
        assert f(d(dt=2)) == -4 and f(d(res=5)) == -4 and f(d(dt=1, res=0)) == -3
        for eps in (-1e-6, float("nan"), float("inf")):
            assert f(d(), eps=eps) == -3
    for kw in (dict(group=64), dict(group=-1), dict(x=M), dict(res=M), dict(w=M), dict(q=M), dict(r=M)):
        assert q8(D(), **kw) == -3
    assert q8(D(C=200)) == -3
    assert bwd(D()) == -5 and bwd(D(ws=P, n=need - 1)) == -5 and bwd(D(ws=M, n=need)) == -3
    assert fwd(D(rows=0), x=None, y=None, r=None) == 0 and q8(D(rows=0), q=None, s=None) == 0
    assert L.kda_add_norm_bwd_workspace_size(None) == 0 and L.kda_add_norm_bwd_workspace_size(ref(D(C=0))) == 0


def test_binding_refusals():
    from gated_delta_rule_63_amd import _layers as M
    z = torch.zeros
    x, w = z(2, 3, 256), z(256)
    ok = lambda x=x, res=x, w=w: M._check_norm(x, res, w, _device=False)
    ok()
    ok(res=None)
    ok(x=x.bfloat16())
    ok(x=x.bfloat16(), res=x.bfloat16())
    for kw in (dict(x=x.half()), dict(res=x.bfloat16()), dict(res=z(6, 256)), dict(w=z(255)), dict(w=w.bfloat16()),
               dict(x=z(2, 3, 0)), dict(x=z(256, 3).T), dict(res=z(2, 256, 3).transpose(1, 2))):
        with pytest.raises(ValueError):
            ok(**kw)
    back = lambda r=x, w=w, dy=x, dr=x: M._check_norm_bwd(r, w, dy, dr, _device=False)
    back()
    back(dy=x.bfloat16(), dr=None)
    for kw in (dict(dr=x.bfloat16()), dict(dr=z(6, 256)), dict(dy=x.half()), dict(r=x.bfloat16())):
        with pytest.raises(ValueError):
            back(**kw)
    with pytest.raises(ValueError):
        ok(x=x, w=w) and M._check_norm(x, x, w)         # not on a GPU


def test_workspace_size():
    import gated_delta_rule_63_amd as kda
    for shape, dtype in (((3, 256), torch.float32), ((2, 5, 7), torch.bfloat16), ((4000, 4096), torch.bfloat16), ((0, 64), torch.float32), ((9,), torch.float32)):
        dy = torch.empty(shape, dtype=dtype)
        d = kda._lib.NormDesc(dy.numel() // shape[-1], shape[-1], 0, 0, None, 0)
        need = kda.add_norm_bwd_workspace_size(dy)
        assert need == kda.lib().kda_add_norm_bwd_workspace_size(ctypes.byref(d)) and (need > 0) == (dy.numel() > 0)
    for bad in (torch.tensor(1.0), torch.empty(3, 0)):
        with pytest.raises(ValueError):
            kda.add_norm_bwd_workspace_size(bad)


def test_outputs_in_the_place_of_inputs():
    """An output exactly where an input lies, or apart from all of them and from the other one."""
    from gated_delta_rule_63_amd import _layers as M
    x, res, w = torch.zeros(4, 64), torch.zeros(4, 64), torch.zeros(64)
    ok = lambda x=x, res=res, w=w, out=None, rout=None: M._check_norm_out(x, res, w, out, rout, _device=False)
    ok()
    ok(out=x, rout=res)
    ok(out=res)
    ok(rout=x)
    ok(out=torch.zeros(4, 64), rout=torch.zeros(4, 64))
    ok(res=None, out=x)
    five = torch.zeros(5, 64)
    half, wide = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64)
    for kw in (dict(out=res, rout=res), dict(out=x, rout=x), dict(x=five[:4], out=five[1:]), dict(res=five[:4], rout=five[1:]),
               dict(res=five[1:], out=five[:4]), dict(w=five[0], out=five[:4]), dict(w=five[3], rout=five[:4]),
               dict(x=half, res=wide, out=wide.view(torch.bfloat16).flatten()[:256].view(4, 64)), dict(res=None, rout=torch.zeros(4, 64))):
        with pytest.raises(ValueError):
            ok(**kw)
    none = torch.zeros(0, 64)
    ok(x=none, res=none, out=none, rout=none)
    with pytest.raises(ValueError):
        M._check_norm_bwd(None, w, x, None, _device=False)


def test_sizes_beyond_32_bits():
    """Rows of 2^32 + 8 channels are refused, not taken for 8. (Tensors without storage.)"""
    from gated_delta_rule_63_amd import _layers as M
    e = lambda *s: torch.empty(*s, device="meta")
    n = (1 << 32) + 8
    with pytest.raises(ValueError, match="32 bits"):
        M._check_norm(e(1, n), None, e(n), _device=False)
    with pytest.raises(ValueError, match="32 bits"):
        M.add_norm_bwd_workspace_size(e(1, n))


# ------------------------------------------------------------------------- GPU

@pytest.fixture
def kda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_63_amd as kda
    return kda


def make(rows, C, dtype, res, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    dt = getattr(torch, dtype)
    rt = None if res is None else getattr(torch, res)
    x, r = n(rows, C).to(dt), 3 * n(rows, C)
    if rows > 2:
        x[1], r[1] = 0.0, 0.0                                # an empty row
        r[2] *= 1e4
    return x, None if rt is None else r.to(rt), 1 + 0.3 * n(C), n(rows, C).to(dt), n(rows, C).to(rt or dt)


SHAPES = [(1, 1), (3, 7), (5, 8), (37, 64), (2, 100), (130, 128), (9, 512), (3, 520), (4, 1000), (33, 2048), (3, 2049), (5, 4096),
          (2, 4104), (3, 8192), (2, 8200), (2, 12288), (1, 16384), (2, 9001), (3, 16383), (700, 136), (301, 100), (67, 250), (9, 256), (65, 1024), (130, 600), (3, 1002), (5, 9004), (2, 4098)]
TYPES = [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32"), ("bfloat16", None), ("float32", None)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_add_norm(kda, rows, C, dtype, res):
    x, r0, w, _, _ = make(rows, C, dtype, res, 1)
    r, r64 = stream(x, r0)
    y, rr = kda.add_norm(x.cuda(), None if r0 is None else r0.cuda(), w.cuda(), eps=EPS)
    torch.cuda.synchronize()
    assert y.dtype == x.dtype and torch.equal(rr.cpu(), r)
    want = norm(r64, w.double().numpy())
    R.held(as64(y), want, rel(C) * np.abs(want), "y", dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_add_norm_q8(kda, rows, C, dtype, res):
    x, r0, w, _, _ = make(rows, C, dtype, res, 2)
    r, r64 = stream(x, r0)
    want = norm(r64, w.double().numpy())
    for group in (0, 128) if C % 128 == 0 else (0,):
        q, scale, rr = kda.add_norm_q8(x.cuda(), None if r0 is None else r0.cuda(), w.cuda(), group=group, eps=EPS)
        torch.cuda.synchronize()
        assert q.dtype == torch.float8_e4m3fn and torch.equal(rr.cpu(), r)
        part = want.reshape(rows, -1, group or C)
        s = np.maximum(np.abs(part).max(-1), 2.0 ** -40) / 448
        assert scale.shape == ((rows, C // 128) if group else (rows,))
        R.held(as64(scale), s if group else s[:, 0], (rel(C) + R.U) * (s if group else s[:, 0]), f"scales {group}")
        # the value lies within rounding of y / scale, so q between what the ends of that range round to
        exact, off = (part / s[..., None]).reshape(rows, C), 2 * rel(C) + 4 * R.U
        to8 = lambda v: torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
        lo, hi = to8(exact - off * np.abs(exact)), to8(np.clip(exact + off * np.abs(exact), -448, 448))
        got = q.float().cpu().double().numpy()
        assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi))), (rows, C, group)
        assert np.all(np.abs(got) <= 448)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,res", TYPES)
@pytest.mark.parametrize("rows,C", SHAPES)
def test_add_norm_bwd(kda, rows, C, dtype, res):
    x, r0, w, dy, dr = make(rows, C, dtype, res, 3)
    r, r64 = stream(x, r0)
    for given in (True, False):
        dx, dres, dw = kda.add_norm_bwd(r.cuda(), w.cuda(), dy.cuda(), dr=dr.cuda() if given else None, eps=EPS)
        torch.cuda.synchronize()
        d, want, bd, bw = grad(r64, w.double().numpy(), dy.double().numpy(), dr.double().numpy() if given else 0.0)
        assert dx.dtype == dy.dtype and dres.dtype == r.dtype
        R.held(as64(dx), d, bd, "dx", dtype)
        R.held(as64(dres), d, bd, "dres", str(r.dtype)[6:])
        R.held(as64(dw), want, bw, "dw")


@pytest.mark.gpu
def test_many_rows(kda):
    """More rows than a launch has workgroups for one each, and the sums over them."""
    rows, C = 150_001, 24
    x, r0, w, dy, dr = make(rows, C, "float32", "float32", 4)
    r, r64 = stream(x, r0)
    y, _ = kda.add_norm(x.cuda(), r0.cuda(), w.cuda(), eps=EPS)
    dx, _, dw = kda.add_norm_bwd(r.cuda(), w.cuda(), dy.cuda(), dr=dr.cuda(), eps=EPS)
    torch.cuda.synchronize()
    want = norm(r64, w.double().numpy())
    R.held(as64(y), want, rel(C) * np.abs(want), "y")
    d, sums, bd, bw = grad(r64, w.double().numpy(), dy.double().numpy(), dr.double().numpy())
    R.held(as64(dx), d, bd, "dx")
    R.held(as64(dw), sums, bw, "dw", rms=1e-5)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 256, 1000, 1002, 1004, 2048, 9008])
@pytest.mark.parametrize("mib", [300, 700])
@pytest.mark.parametrize("dtype,res", TYPES)
def test_calls_beyond_the_cache(kda, dtype, res, mib, C):
    """Rows of large calls have the bits of the same rows in small ones; dweight from the few rows
    that add to it."""
    dt, rt = getattr(torch, dtype), getattr(torch, res or dtype)
    e, re = dt.itemsize, rt.itemsize
    gen = torch.Generator("cuda").manual_seed(5)
    many = lambda n, t: torch.empty(n, C, dtype=t, device="cuda").normal_(generator=gen)
    w = 1 + 0.3 * many(1, torch.float32)[0]
    for part, size in (("y", e + e + (2 * re if res else 0)), ("q8", e + 1 + (2 * re if res else 0)), ("bwd", 2 * e + 3 * re)):
        n = (mib << 20) // (size * C)
        x = many(n, dt)
        r0 = many(n, rt) if res or part == "bwd" else None
        places = [slice(0, 70), slice(n // 2 - 35, n // 2 + 35), slice(n - 70, n)]
        cut = lambda t, at: None if t is None else t[at].clone()
        if part == "bwd":
            x[torch.arange(n, device="cuda") % 97 != 5] = 0
            dr = many(n, rt)
            dx, dres, dw = kda.add_norm_bwd(r0, w, x, dr=dr, eps=EPS)
            used = slice(5, None, 97)
            want, _, bw = grad(as64(r0[used]), as64(w), as64(x[used]), 0.0)[1:]
            R.held(as64(dw), want, bw, "dw")
            for at in places:
                for got, small in zip((dx, dres), kda.add_norm_bwd(cut(r0, at), w, cut(x, at), dr=cut(dr, at), eps=EPS)):
                    assert torch.equal(got[at], small)
        else:
            call = kda.add_norm if part == "y" else kda.add_norm_q8
            got = call(x, r0, w, eps=EPS)
            for at in places:
                for whole, small in zip(got, call(cut(x, at), cut(r0, at), w, eps=EPS)):
                    view = (lambda t: t.view(torch.uint8)) if whole.dtype.itemsize == 1 else (lambda t: t)
                    assert torch.equal(view(whole[at]), view(small))


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 4096, 4101])
def test_in_place_unaligned_and_no_rows(kda, C):
    """Outputs in the place of inputs, tensors that start on no 16 bytes, and calls without rows."""
    x, r0, w, dy, dr = (t.cuda() for t in make(6, C, "bfloat16", "bfloat16", 5))
    y, r = kda.add_norm(x, r0, w)
    d, _, dw = kda.add_norm_bwd(r, w, dy, dr=dr)
    q, s, _ = kda.add_norm_q8(x, r0, w)
    xi, ri = x.clone(), r0.clone()
    got = kda.add_norm(xi, ri, w, out=xi, residual_out=ri)
    assert got[0] is xi and got[1] is ri and torch.equal(xi, y) and torch.equal(ri, r)
    flat = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].reshape(t.shape)
    ux, ur, udy, udr = flat(x), flat(r0), flat(dy), flat(dr)
    assert ux.data_ptr() % 16 and ux.is_contiguous()
    uy, urr = kda.add_norm(ux, ur, w)
    # the sums are ordered otherwise: a step of bf16 where a value lies between two
    assert torch.equal(urr, r) and float((uy.float() - y.float()).abs().max()) <= 2.0 ** -7 * float(y.abs().max())
    ud, _, udw = kda.add_norm_bwd(flat(r), w, udy, dr=udr)
    assert float((ud.float() - d.float()).abs().max()) <= 2.0 ** -7 * float(d.abs().max())
    assert float((udw - dw).abs().max()) <= 1e-5 * float(dw.abs().max())
    uq, us, _ = kda.add_norm_q8(ux, ur, w)
    assert float((us - s).abs().max()) <= 2 * rel(C) * float(s.max())
    assert float((uq.float() - q.float()).abs().max()) <= 32                       # a step at 448
    none = x[:0]
    y0, r0_ = kda.add_norm(none, none, w)
    d0, _, dw0 = kda.add_norm_bwd(none, w, none)
    q0, s0, _ = kda.add_norm_q8(none, None, w)
    assert y0.shape == r0_.shape == d0.shape == q0.shape == (0, C) and s0.shape == (0,) and not bool(dw0.any())


@pytest.mark.gpu
def test_rows_that_are_not_numbers(kda):
    """A row with an infinity or NaN touches no other row."""
    x, r0, w, _, _ = (t.cuda() for t in make(5, 640, "float32", "float32", 6))
    y, r = kda.add_norm(x, r0, w)
    q, s, _ = kda.add_norm_q8(x, r0, w, group=128)
    x[1, 3], x[3, 600] = float("inf"), float("nan")
    y2, r2 = kda.add_norm(x, r0, w)
    q2, s2, _ = kda.add_norm_q8(x, r0, w, group=128)
    for i in (0, 2, 4):
        assert torch.equal(y2[i], y[i]) and torch.equal(r2[i], r[i])
        assert torch.equal(q2[i].view(torch.uint8), q[i].view(torch.uint8)) and torch.equal(s2[i], s[i])
    assert bool(y2[1, 3].isnan()) and bool(y2[3].isnan().all())


@pytest.mark.gpu
def test_streams_and_graphs(kda):
    x, r0, w, dy, dr = (t.cuda() for t in make(300, 2048, "bfloat16", "float32", 7))

    def both(stream=None):
        y, r = kda.add_norm(x, r0, w, stream=stream)
        return (y, r, *kda.add_norm_q8(x, r0, w, group=128, stream=stream)[:2],
                *kda.add_norm_bwd(r, w, dy, dr=dr, stream=stream))

    same = lambda a, b: all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))
    want = both()
    torch.cuda.synchronize()
    got = [both(st) for st in (torch.cuda.Stream(), torch.cuda.Stream())]
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(3):
        for u in held:
            u.view(torch.uint8).fill_(1)
        graph.replay()
        other = both()
        torch.cuda.synchronize()
        assert same(held, want) and same(other, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,res", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "float32")])
@pytest.mark.parametrize("C", [8, 100, 128, 200, 256, 600, 1000, 1024, 1025, 2048])
def test_eps_of_zero(kda, C, dtype, res, monkeypatch):
    """eps = 0 over rows that are not zero, at numbers of rows that fill a workgroup or do not."""
    monkeypatch.setitem(globals(), "EPS", 0.0)              # of the references
    gen = torch.Generator().manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=gen)
    dt, rt = getattr(torch, dtype), getattr(torch, res)
    for rows in (1, 4, 7, 9, 16, 17):
        x, r0, w, dy, dr = n(rows, C).to(dt), (3 * n(rows, C)).to(rt), 1 + 0.3 * n(C), n(rows, C).to(dt), n(rows, C).to(rt)
        r, r64 = stream(x, r0)
        y, rr = kda.add_norm(x.cuda(), r0.cuda(), w.cuda(), eps=0.0)
        dx, dres, dw = kda.add_norm_bwd(r.cuda(), w.cuda(), dy.cuda(), dr=dr.cuda(), eps=0.0)
        torch.cuda.synchronize()
        want = norm(r64, w.double().numpy())
        assert torch.equal(rr.cpu(), r)
        R.held(as64(y), want, rel(C) * np.abs(want), f"y, {rows} rows", dtype)
        d, sums, bd, bw = grad(r64, w.double().numpy(), dy.double().numpy(), dr.double().numpy())
        R.held(as64(dx), d, bd, "dx", dtype)
        R.held(as64(dres), d, bd, "dres", res)
        R.held(as64(dw), sums, bw, f"dw, {rows} rows")


@pytest.mark.gpu
def test_in_place_without_a_residual(kda):
    """The norm in x's place leaves no sum to return; elsewhere x is the sum."""
    x, _, w, dy, _ = (t.cuda() for t in make(5, 200, "float32", "float32", 9))
    y, r = kda.add_norm(x, None, w)
    assert r is x and kda.add_norm(x[:0], None, w)[1].shape == (0, 200)
    xi = x.clone()
    got, lost = kda.add_norm(xi, None, w, out=xi)
    assert got is xi and lost is None and torch.equal(got, y)
    with pytest.raises(ValueError):
        kda.add_norm_bwd(lost, w, dy)
    with pytest.raises(ValueError):
        kda.add_norm(x, x, w, out=xi, residual_out=xi)


@pytest.mark.gpu
def test_given_workspace(kda):
    """Of the size that is asked for; a byte less is refused."""
    x, r0, w, dy, dr = (t.cuda() for t in make(70, 640, "bfloat16", "float32", 10))
    want = kda.add_norm_bwd(r0, w, dy, dr=dr)
    need = kda.add_norm_bwd_workspace_size(dy)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(kda.add_norm_bwd(r0, w, dy, dr=dr, workspace=ws), want))
    with pytest.raises(kda.KDAError):
        kda.add_norm_bwd(r0, w, dy, dr=dr, workspace=ws[:need - 1])
    with pytest.raises(ValueError):
        kda.add_norm_bwd(r0, w, dy, dr=dr, workspace=ws.cpu())

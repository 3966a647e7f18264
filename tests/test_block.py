"""What comes before and after the rule (kda_block_in, kda_block_out, their Gated
DeltaNet forms and gradients) against the formulas in 64 bits, whose gradients
come from torch's differentiation and, once, from differences; and the whole
block, forwards and backwards."""
import ctypes

import numpy as np
import pytest

from ops_ref import rule_bwd, within

torch = pytest.importorskip("torch")
P, M = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)   # never dereferenced


def block_in(q, k, f, b, A, bias, bound, eps):
    unit = lambda u: u / (u.square().sum(-1, keepdim=True) + eps).sqrt()
    a = A.exp() if f.dim() == 3 else A.exp()[:, None]
    x = f if bias is None else f + bias
    g = -a * torch.logaddexp(x, torch.zeros_like(x)) if bound is None else bound * torch.sigmoid(a * x)
    return unit(q), unit(k), g, torch.sigmoid(b)


def block_out(o, z, w, act, eps):
    s = torch.sigmoid(z)
    return o / (o.square().mean(-1, keepdim=True) + eps).sqrt() * w * (s if act == "sigmoid" else z * s)


def grads(f, leaves, up):
    leaves = [None if x is None else x.detach().double().requires_grad_() for x in leaves]
    y = f(*leaves)
    y = y if isinstance(y, tuple) else (y,)
    on = [x for x in leaves if x is not None]
    got = iter(torch.autograd.grad(y, on, [u.double() for u in up]))
    return y, [None if x is None else next(got) for x in leaves]


# ------------------------------------------------------------------------- CPU

def test_reference_gradients_against_differences():
    gen = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)
    for fn, leaves in (
            (lambda *x: block_in(*x, None, 1e-6), [n(2, 3, 2, 8), n(2, 3, 2, 8), n(2, 3, 2, 8), n(2, 3, 2), n(2), n(2, 8)]),
            (lambda *x: block_in(*x, -5.0, 1e-6), [n(2, 3, 2, 8), n(2, 3, 2, 8), n(2, 3, 2), n(2, 3, 2), n(2), n(2)]),
            (lambda *x: block_out(*x, "sigmoid", 1e-5), [n(2, 3, 2, 8), n(2, 3, 2, 8), n(8)]),
            (lambda *x: block_out(*x, "silu", 1e-5), [n(2, 3, 2, 8), n(2, 3, 2, 8), n(8)])):
        torch.autograd.gradcheck(fn, [x.requires_grad_() for x in leaves])


def test_refusals():
    import gated_delta_rule_63_amd as kda
    L = kda.lib()

    def desc(B=2, T=3, H=2, K=128, dt=0, N=None, ws=1 << 30):
        return ctypes.byref(kda.Desc(B, T, H, K, 128, B if N is None else N, dt, 1, P if ws else None, ws))

    for pre in ("kda_", "kda_gdn_"):
        names = "q k f b A bias".split(), "qo ko g beta".split(), "dqo dko dg dbeta dq dk df db dA dbias".split()

        def call(bwd, bound=0.0, eps=1e-6, d=None, **kw):
            a = {n: kw.get(n, P) for n in names[0]}
            r = {n: kw.get(n, P) for n in names[2 if bwd else 1]}
            fn = getattr(L, pre + ("block_in_bwd" if bwd else "block_in"))
            return fn(*a.values(), bound, eps, *r.values(), d or desc(), None)

        wide = [n for n in ("q", "k", "f", "bias", "g", "qo", "ko") if pre == "kda_" or n not in ("f", "bias", "g")]
        for n in ("q", "k", "f", "b", "A", "qo", "ko", "g", "beta"):
            assert call(False, **{n: None}) == -1, n
        for n in wide:
            assert call(False, **{n: M}) == -3, n
        for n in ("dqo", "dko", "dg", "dbeta", "dq", "dk", "df", "db", "dA"):
            assert call(True, **{n: None}) == -1, n
        for bad in (1.0, float("nan"), float("-inf")):
            assert call(False, bound=bad) == -3 and call(True, bound=bad) == -3
        for bad in (-1e-6, float("nan"), float("inf")):
            assert call(False, eps=bad) == -3 and call(True, eps=bad) == -3
        assert call(True, d=desc(ws=0)) == -5 and call(True, d=desc(ws=4)) == -5
        assert call(False, d=desc(K=64)) == -3 and call(False, d=desc(dt=9)) == -4 and call(False, d=desc(T=-1)) == -2
        assert call(False, d=desc(B=1 << 15, T=1 << 15)) == -2          # 2^31 rows
        assert call(True, d=desc(B=1 << 14, T=1 << 13, H=2)) == -2       # 2^28

    def out(bwd, act=0, eps=1e-5, d=None, **kw):
        a = {n: kw.get(n, P) for n in "o z w".split()}
        r = {n: kw.get(n, P) for n in ("dy do dz dw".split() if bwd else ["y"])}
        return getattr(L, "kda_block_out_bwd" if bwd else "kda_block_out")(*a.values(), eps, act, *r.values(),
                                                                            d or desc(), None)
    for n in ("o", "z", "w", "y"):
        assert out(False, **{n: None}) == -1 and out(False, **{n: M}) == -3
    for n in ("dy", "do", "dz"):
        assert out(True, **{n: None}) == -1 and out(True, **{n: M}) == -3
    assert out(True, dw=None) == -1 and out(False, act=2) == -3 and out(False, eps=-1.0) == -3
    assert out(True, d=desc(ws=0)) == -5 and out(False, d=desc(K=64)) == -3
    assert out(False, d=desc(T=0), o=None, z=None, y=None) == 0


def test_binding_refusals():
    from gated_delta_rule_63_amd import _ops
    z = torch.zeros
    q, b, A, bias = z(2, 3, 4, 128), z(2, 3, 4), z(4), z(4, 128)

    def ok(q=q, k=q, f=q, b=b, A=A, bias=bias, bound=None, s=False, dq=q, dk=q, dg=q, db=b):
        _ops._check_block_in_bwd(q, k, f, b, A, dq, dk, dg, db, bias, bound, s, _device=False)

    ok()
    ok(bound=-5.0, bias=None)
    ok(f=b, bias=z(4), dg=b, s=True)
    for kw in (dict(bound=-1e-50), dict(q=q.half()), dict(k=q.bfloat16()), dict(f=b), dict(b=z(2, 3)), dict(A=z(3)), dict(bias=z(4)),
               dict(bound=5.0), dict(bound=0.0), dict(dg=q.bfloat16()), dict(dq=z(2, 3, 4, 64)),
               dict(k=z(2, 3, 128, 4).transpose(2, 3))):
        with pytest.raises(ValueError):
            ok(**kw)
    out = lambda o=q, z=q, w=z(128), act="silu", dy=q: _ops._check_block_out(o, z, w, act, dy, _device=False)
    out()
    out(z=q.bfloat16(), dy=q.bfloat16())
    for kw in (dict(o=q.bfloat16()), dict(z=q.half()), dict(w=z(64)), dict(act="relu"), dict(dy=q.bfloat16()),
               dict(w=z(128).bfloat16())):
        with pytest.raises(ValueError):
            out(**kw)


# ------------------------------------------------------------------------- GPU

@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def held(got, ref, what):
    """bf16 results are off by half a step of their type. An fp32 result far above the
    RMS (a gate of 100 on a row of one channel: 1e3 against 5) is off by its own
    rounding: a product of at most eight factors (n: a sum, a root, a division and a
    product; w; act: an exponential and a reciprocal of two half steps each, a sum and
    a product), so at most 16 half steps of 2^-24 relative to it, 2^-20."""
    within(got.float().cpu().numpy(), ref.detach().numpy(), what, 2.0 ** (-8 if got.dtype == torch.bfloat16 else -20), tol=2e-5)


SHAPES = [(1, 1, 1), (3, 5, 1), (1, 17, 3), (2, 67, 16), (1, 9, 17), (1, 300, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scalar,bound,bias", [(False, None, True), (False, -5.0, False), (True, None, False), (True, -2.5, True)])
def test_block_in(gpu, B, T, H, dtype, scalar, bound, bias):
    import gated_delta_rule_63_amd as kda
    gen = torch.Generator().manual_seed(B * T + H)
    n = lambda *s: torch.randn(*s, generator=gen)
    gate = (B, T, H) if scalar else (B, T, H, 128)
    q, k, f, b = n(B, T, H, 128).to(dtype), (30 * n(B, T, H, 128)).to(dtype), (3 * n(*gate)).to(dtype), (4 * n(B, T, H)).to(dtype)
    f.view(-1)[:2] = torch.tensor([60.0, -60.0], dtype=dtype)[:f.numel()]   # the gate's flat ends
    b.view(-1)[0] = -80.0
    q[0, 0, 0] = 0.0                                           # a row without a direction
    A, bb = torch.rand(H, generator=gen), (n(*gate[2:]) if bias else None)
    up = [n(B, T, H, 128).to(dtype), n(B, T, H, 128).to(dtype), n(*gate), n(B, T, H)]
    ref, want = grads(lambda *x: block_in(*x, bound, 1e-6), [q, k, f, b, A, bb], up)
    c = lambda x: None if x is None else x.cuda()
    pre = "gdn_" if scalar else ""
    y = getattr(kda, pre + "block_in")(*map(c, (q, k, f, b, A)), dt_bias=c(bb), lower_bound=bound)
    for x, r, name in zip(y, ref, "q k g beta".split()):
        held(x, r, name)
    d = getattr(kda, pre + "block_in_bwd")(*map(c, (q, k, f, b, A, *up)), dt_bias=c(bb), lower_bound=bound)
    # the row of zeros divides by sqrt(eps): its gradient is 1e3 times the others', and is held by itself
    for x, r, name in zip(d, want, "dq dk df db dA dbias".split()):
        if name == "dq":
            held(x[0, 0, 0], r[0, 0, 0], "dq of zero")
            x, r = x.reshape(-1, 128)[1:], r.reshape(-1, 128)[1:]
        if r is not None:
            held(x, r, name)
    assert (d[5] is None) == (bb is None)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,H", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_block_out(gpu, B, T, H, dtype, act):
    import gated_delta_rule_63_amd as kda
    gen = torch.Generator().manual_seed(B * T + H)
    n = lambda *s: torch.randn(*s, generator=gen)
    o, z, w, dy = n(B, T, H, 128), (4 * n(B, T, H, 128)).to(dtype), n(128), n(B, T, H, 128).to(dtype)
    o[0, 0, 0, 1:] = 0.0                                       # one channel alone
    o[-1, -1, -1] *= 1e-4                                      # a row as small as eps
    z.view(-1)[:2] = torch.tensor([100.0, -100.0], dtype=dtype)
    (ref,), want = grads(lambda *x: block_out(*x, act, 1e-5), [o, z, w], [dy])
    held(kda.block_out(o.cuda(), z.cuda(), w.cuda(), activation=act), ref, "y")
    got = kda.block_out_bwd(o.cuda(), z.cuda(), w.cuda(), dy.cuda(), activation=act)
    # do is the difference r dn - r n mean(n dn), whose two terms nearly cancel in the
    # row of one channel: each is rounded by at most 16 half steps of its own size
    with torch.no_grad():
        od, zd = o.double(), z.double()
        r = (od.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
        dn = dy.double() * w.double() * torch.sigmoid(zd) * (zd if act == "silu" else 1.0)
        terms = 2.0 ** -20 * (r * (dn.abs() + (od * r).abs() * (od * r * dn).abs().mean(-1, keepdim=True))).numpy()
    f = lambda x: x.detach().cpu().reshape(-1, 128).double().numpy()
    # the small row's do is about 300 times the others': by itself
    within(f(got[0])[-1], f(want[0])[-1], "do of the small row", terms.reshape(-1, 128)[-1], tol=2e-5)
    if B * T * H > 1:
        within(f(got[0])[:-1], f(want[0])[:-1], "do", terms.reshape(-1, 128)[:-1], tol=2e-5)
    held(got[1], want[1], "dz")
    held(got[2], want[2], "dw")


@pytest.mark.gpu
def test_no_tokens(gpu):
    """T = 0: empty outputs, and sums over nothing are zero."""
    import gated_delta_rule_63_amd as kda
    e = lambda *s: torch.zeros(*s, device="cuda")
    q, b, A, bias = e(2, 0, 3, 128), e(2, 0, 3), e(3), e(3, 128) + 1.0
    assert all(x.numel() == 0 for x in kda.block_in(q, q, q, b, A, dt_bias=bias))
    got = kda.block_in_bwd(q, q, q, b, A, q, q, q, b, dt_bias=bias)
    assert not bool(got[4].any()) and not bool(got[5].any())
    assert kda.block_out(q, q, e(128)).numel() == 0 and not bool(kda.block_out_bwd(q, q, e(128), q)[2].any())


@pytest.mark.gpu
def test_far_rows(gpu):
    """Rows whose elements lie beyond 2^31 are those of a call on them alone."""
    import gated_delta_rule_63_amd as kda
    gen = torch.Generator(device="cuda").manual_seed(9)
    T, H, m = 140000, 120, 7
    assert T * H * 128 > 2 ** 31
    def tail(dtype, *s):
        x = torch.zeros(1, T, *s, dtype=dtype, device="cuda")
        x[:, -m:] = torch.randn(1, m, *s, generator=gen, device="cuda").to(dtype)
        return x
    q, f, b, g, db = (tail(torch.bfloat16, H, 128), tail(torch.bfloat16, H, 128), tail(torch.bfloat16, H),
                      tail(torch.float32, H, 128), tail(torch.float32, H))
    A, w = torch.rand(H, generator=gen, device="cuda"), torch.rand(128, generator=gen, device="cuda")
    last = lambda x: x[:, -m:].contiguous()
    for fn, args, rest in ((kda.block_in, (q, q, f, b), (A,)), (kda.block_out, (g, q), (w,)),
                           (lambda *x: kda.block_in_bwd(*x[:4], A, *x[4:])[:4], (q, f, f, b, f, q, g, db), ()),
                           (lambda *x: kda.block_out_bwd(*x[:2], w, x[2])[:2], (g, q, f), ())):
        got, want = fn(*args, *rest), fn(*map(last, args), *rest)
        if torch.is_tensor(got):
            got, want = [got], [want]
        assert all(torch.equal(x[:, -m:], y) for x, y in zip(got, want))
        del got, want


@pytest.mark.gpu
def test_in_place(gpu):
    """What include/kda.h allows to share memory does."""
    import gated_delta_rule_63_amd as kda
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    B, T, H = 2, 65, 5
    q, k, f, b, A, o, z, w, dy = (n(B, T, H, 128), n(B, T, H, 128), n(B, T, H, 128), n(B, T, H), n(H), n(B, T, H, 128),
                                  n(B, T, H, 128), n(128), n(B, T, H, 128))
    want = kda.block_in(q, k, f, b, A), kda.block_out_bwd(o, z, w, dy)
    g, beta, dw, ws = torch.empty_like(f), torch.empty_like(b), torch.empty_like(w), torch.empty(1 << 20, device="cuda")
    d = kda.Desc(B, T, H, 128, 128, B, 1, 1, ws.data_ptr(), ws.numel() * 4)
    p = lambda x: ctypes.c_void_p(x.data_ptr())
    L = kda.lib()
    assert L.kda_block_in(p(q), p(k), p(f), p(b), p(A), None, 0.0, 1e-6, p(q), p(k), p(g), p(beta), ctypes.byref(d), None) == 0
    assert L.kda_block_out_bwd(p(o), p(z), p(w), 1e-5, 0, p(dy), p(o), p(dy), p(dw), ctypes.byref(d), None) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((q, k, g, beta, o, dy, dw), (*want[0], *want[1])))


@pytest.mark.gpu
def test_same_bits_on_streams_and_in_graphs(gpu):
    import gated_delta_rule_63_amd as kda
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    B, T, H = 1, 400, 24
    q, f, b, A, bias, g, o, w = n(B, T, H, 128), n(B, T, H, 128), n(B, T, H), n(H), n(H, 128), n(B, T, H, 128), n(B, T, H, 128), n(128)
    run = lambda **k: (*kda.block_in_bwd(q, f, f, b, A, g, o, g, b, dt_bias=bias, **k), *kda.block_out_bwd(o, q, w, g, **k),
                       *kda.block_in(q, f, f, b, A, dt_bias=bias, **k), kda.block_out(o, q, w, **k))
    first = run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = run(stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    for rep in range(3):
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, out)), rep
        n(1000).sum()


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_whole_block(gpu, scalar, dtype):
    """Norms and gates, the rule, the gated norm, and the gradients back through all
    three. Every step against the formula in 64 bits at the inputs that the step
    before it left, to that step's own bar (the rule forwards: 2e-2 of its RMS in bf16,
    1e-4 in fp32). In fp32 the ends are also compared with the block in 64 bits as a
    whole: three steps back and one forwards at 1e-4 each. (In bf16 that has no bar:
    the norm divides a row by its own size, and with it the rounding of q and k, which
    does not follow the size of the row that q and k give.)"""
    import gated_delta_rule_63_amd as kda
    B, T, H = 2, 75, 3
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen)
    gate = (B, T, H) if scalar else (B, T, H, 128)
    q, k, v, z, dy = (n(B, T, H, 128).to(dtype) for _ in range(5))
    f, b = n(*gate).to(dtype), n(B, T, H).to(dtype)
    A, bias, w = torch.rand(H, generator=gen), n(*gate[2:]), 1 + 0.1 * n(128)
    c = lambda *x: [t.cuda() for t in x]
    pre = "gdn_" if scalar else ""
    gq, gk, gv, gz, gdy, gf, gb, gA, gbias, gw = c(q, k, v, z, dy, f, b, A, bias, w)
    ins = getattr(kda, pre + "block_in")(gq, gk, gf, gb, gA, dt_bias=gbias, lower_bound=-5.0)
    q1, k1, g1, b1 = ins
    o, _ = getattr(kda, pre + "fwd")(q1, k1, gv, g1, b1)
    y = kda.block_out(o, gz, gw, activation="silu")
    do, dz, dw = kda.block_out_bwd(o, gz, gw, gdy, activation="silu")
    d = getattr(kda, pre + "bwd")(q1, k1, gv, g1, b1, do)
    got = getattr(kda, pre + "block_in_bwd")(gq, gk, gf, gb, gA, d[0], d[1], d[3], d[4], dt_bias=gbias, lower_bound=-5.0)

    def rule(q, k, v, g, b):
        S, out = torch.zeros(B, H, 128, 128, dtype=torch.float64), []
        for t in range(T):
            S = (g[:, t, :, None] if scalar else g[:, t]).exp()[..., None] * S
            e = v[:, t] - (S * k[:, t, ..., None]).sum(-2)
            S = S + k[:, t, ..., None] * (b[:, t, :, None] * e)[..., None, :]
            out.append((S * q[:, t, ..., None]).sum(-2))
        return torch.stack(out, 1)

    back = lambda *x: [torch.from_numpy(u) for u in rule_bwd(*(t.double().numpy() for t in x), [(i, 0, T) for i in range(B)])]
    f_in, f_out = lambda *u: block_in(*u, -5.0, 1e-6), lambda *u: block_out(*u, "silu", 1e-5)
    cpu = lambda x: [t.detach().cpu().double() for t in x]
    np_ = lambda x: x.detach().float().cpu().numpy() if x.dtype == torch.bfloat16 else x.detach().cpu().numpy()
    half = lambda x: 2.0 ** (-8 if x.dtype == torch.bfloat16 else -20)

    # step by step
    ref, want = grads(f_in, [q, k, f, b, A, bias], cpu([d[0], d[1], d[3], d[4]]))
    for name, x, r in [*zip("q k g beta".split(), ins, ref), *zip("dq dk df db dA dbias".split(), got, want)]:
        held(x, r, name)
    within(np_(o), rule(*cpu([q1, k1, gv, g1, b1])).numpy(), "o", tol=2e-2 if dtype == torch.bfloat16 else 1e-4)
    (ry,), (rdo, rdz, rdw) = grads(f_out, [o.cpu(), z, w], [dy])
    for name, x, r in (("y", y, ry), ("dz", dz, rdz), ("dw", dw, rdw), ("do", do, rdo)):
        held(x, r, name)
    for name, x, r in zip("dq' dk' dv dg dbeta".split(), d, back(*cpu([q1, k1, gv, g1, b1, do]))):
        within(np_(x), r.numpy(), name, half(x))
    if dtype == torch.bfloat16:
        return
    # as a whole
    ref = [x.detach() for x in f_in(*cpu([q, k, f, b, A, bias]))]
    r_o = rule(ref[0], ref[1], v.double(), ref[2], ref[3])
    (r_y,), (r_do, r_dz, r_dw) = grads(f_out, [r_o, z, w], [dy])
    r_d = back(ref[0], ref[1], v, ref[2], ref[3], r_do)
    _, r_got = grads(f_in, [q, k, f, b, A, bias], [r_d[0], r_d[1], r_d[3], r_d[4]])
    for name, x, r in [("y", y, r_y), ("dz", dz, r_dz), ("dw", dw, r_dw), ("dv", d[2], r_d[2]),
                       *zip("dq dk df db dA dbias".split(), got, r_got)]:
        within(np_(x), r.detach().numpy(), "whole " + name, tol=4e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
def test_default_gate_into_the_rule(gpu, scalar):
    """The gate without a bound goes below -5 where raw gates are large, and the rule takes
    that as long as such gates are rare (16 tokens sum to more than -80): forwards and
    back, each step to its own bar at the inputs the step before it left."""
    import gated_delta_rule_63_amd as kda
    B, T, H = 1, 90, 2
    gen = torch.Generator().manual_seed(21)
    n = lambda *s: torch.randn(*s, generator=gen)
    gate = (B, T, H) if scalar else (B, T, H, 128)
    f, b = n(*gate), n(B, T, H)
    f[:, 5::12] += 2.5
    q, k, v, do = (n(B, T, H, 128) for _ in range(4))
    c = lambda x: x.cuda()
    pre = "gdn_" if scalar else ""
    q1, k1, g, beta = getattr(kda, pre + "block_in")(c(q), c(k), c(f), c(b), c(torch.full((H,), 1.0)))
    lows = g.unfold(1, 16, 1).sum(-1).min().item()
    assert g.min().item() < -6.0 and lows > -80.0, (g.min().item(), lows)
    o, hT = getattr(kda, pre + "fwd")(q1, k1, c(v), g, beta)
    d = getattr(kda, pre + "bwd")(q1, k1, c(v), g, beta, c(do))
    x = [t.cpu().double().numpy() for t in (q1, k1, c(v), g, beta)]
    S, ref_o = np.zeros((H, 128, 128)), []
    for t in range(T):
        S = np.exp(x[3][0, t])[..., None, None] * S if scalar else np.exp(x[3][0, t])[..., None] * S
        e = x[2][0, t] - np.einsum("hk,hkv->hv", x[1][0, t], S)
        S = S + np.einsum("hk,hv->hkv", x[1][0, t], x[4][0, t][:, None] * e)
        ref_o.append(np.einsum("hk,hkv->hv", x[0][0, t], S))
    within(o[0].cpu().numpy(), np.stack(ref_o), "o")
    within(hT[0].cpu().numpy(), S, "hT")
    for name, u, r in zip("dq dk dv dg dbeta dh0".split(), d, rule_bwd(*x, do.double().numpy(), [(0, 0, T)])):
        within(u.cpu().numpy(), r, name)


@pytest.mark.gpu
def test_two_calls_at_once(gpu):
    """The gradients' partial sums of two calls that run at the same time stay apart."""
    import gated_delta_rule_63_amd as kda
    gen = torch.Generator(device="cuda").manual_seed(6)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    B, T, H = 1, 2048, 16
    q, f, b, A, bias, g, o, w = n(B, T, H, 128), n(B, T, H, 128), n(B, T, H), n(H), n(H, 128), n(B, T, H, 128), n(B, T, H, 128), n(128)
    up = [n(B, T, H, 128), n(B, T, H, 128)]
    run = lambda u, **k: (*kda.block_in_bwd(q, f, f, b, A, u, o, u, b, dt_bias=bias, **k), *kda.block_out_bwd(o, q, w, u, **k))
    alone = [run(u) for u in up]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [run(u, stream=s) for _ in range(3) for u, s in zip(up, streams)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(out, alone[i % 2])), i
    assert not torch.equal(alone[0][4], alone[1][4])


@pytest.mark.gpu
def test_joined_by_autograd_functions(gpu):
    """The calls joined with their gradients in torch.autograd.Function, as the binding
    describes it: a step's gradients are those of the calls made one by one, and stay so
    on a side stream. The calls alone leave no graph."""
    import gated_delta_rule_63_amd as kda

    class In(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, f, b, A, bias):
            ctx.save_for_backward(q, k, f, b, A, bias)
            return kda.block_in(q, k, f, b, A, dt_bias=bias, lower_bound=-5.0)

        @staticmethod
        def backward(ctx, *up):
            *x, bias = ctx.saved_tensors
            return kda.block_in_bwd(*x, *(u.contiguous() for u in up), dt_bias=bias, lower_bound=-5.0)

    class Rule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *x):
            ctx.save_for_backward(*x)
            return kda.fwd(*x, output_final_state=False)[0]

        @staticmethod
        def backward(ctx, do):
            return kda.bwd(*ctx.saved_tensors, do.contiguous())[:5]

    class Out(torch.autograd.Function):
        @staticmethod
        def forward(ctx, o, z, w):
            ctx.save_for_backward(o, z, w)
            return kda.block_out(o, z, w)

        @staticmethod
        def backward(ctx, dy):
            return kda.block_out_bwd(*ctx.saved_tensors, dy.contiguous())

    gen = torch.Generator(device="cuda").manual_seed(31)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    B, T, H = 2, 70, 3
    leaves = [n(B, T, H, 128), n(B, T, H, 128), n(B, T, H, 128), n(B, T, H), 0.3 * n(H), n(H, 128), n(B, T, H, 128),
              n(B, T, H, 128), 1 + 0.1 * n(128)]
    dy = n(B, T, H, 128)
    q, k, f, b, A, bias, v, z, w = leaves
    ins = kda.block_in(q, k, f, b, A, dt_bias=bias, lower_bound=-5.0)
    o = kda.fwd(ins[0], ins[1], v, *ins[2:], output_final_state=False)[0]
    do, dz, dw = kda.block_out_bwd(o, z, w, dy)
    dq, dk, dv, dg, db, _ = kda.bwd(ins[0], ins[1], v, *ins[2:], do)
    want = [*kda.block_in_bwd(q, k, f, b, A, dq, dk, dg, db, dt_bias=bias, lower_bound=-5.0), dv, dz, dw]

    def step():
        x = [t.detach().clone().requires_grad_() for t in leaves]
        q1, k1, g1, b1 = In.apply(*x[:6])
        y = Out.apply(Rule.apply(q1, k1, x[6], g1, b1), *x[7:])
        return torch.autograd.grad((y * dy).sum(), x)

    assert not kda.block_out(o.requires_grad_(), z, w).requires_grad
    side = torch.cuda.Stream()
    got = [step()]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got.append(step())
    torch.cuda.synchronize()
    for grads_ in got:
        assert all(torch.equal(x, y) for x, y in zip(grads_, want))

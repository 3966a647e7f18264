"""The gradient of the chunked rule (kda_bwd, kda_gdn_bwd) against the adjoint of
the token recurrence in fp64, and that adjoint against differences of the forward."""
import ctypes

import numpy as np
import pytest

import workloads as W
from ops_ref import rule_bwd, within

P = ctypes.c_void_p(0x10000)   # never dereferenced


# ------------------------------------------------------------------------- CPU

def _forward(q, k, v, g, beta, do, h0, dhT):
    """sum(o * do) + sum(hT * dhT) of one sequence, by the recurrence in fp64."""
    S, loss = h0.copy(), 0.0
    for t in range(q.shape[0]):
        S = np.exp(g[t])[..., None] * S
        e = v[t] - np.einsum("hk,hkv->hv", k[t], S)
        S = S + np.einsum("hk,hv->hkv", k[t], beta[t][:, None] * e)
        loss += np.sum(np.einsum("hk,hkv->hv", q[t], S) * do[t])
    return loss + np.sum(S * dhT)


@pytest.mark.parametrize("scalar", [False, True])
def test_reference_against_differences(scalar):
    """Central differences along random directions, one input at a time. The loss is
    smooth: with a step of 1e-4 the truncation is about 1e-8 of its third derivative
    and the rounding 1e-16 / 1e-4 of the loss."""
    rng = np.random.default_rng(7)
    T, H, D = 9, 2, 128
    n = lambda *s: rng.standard_normal(s)
    q, k, v, do = (n(T, H, D) for _ in range(4))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    g = -np.abs(n(T, H, 1) if scalar else n(T, H, D))
    beta, h0, dhT = rng.random((T, H)), 0.1 * n(H, D, D), 0.1 * n(H, D, D)
    args = [q, k, v, g, beta, do, h0, dhT]
    got = rule_bwd(q[None], k[None], v[None], g[None, ..., 0] if scalar else g[None], beta[None], do[None],
                   [(0, 0, T)], h0[None], dhT[None])
    for i, grad in zip((0, 1, 2, 3, 4, 6), got):
        step = n(*args[i].shape)
        at = lambda x: _forward(*args[:i], args[i] + x * step, *args[i + 1:])
        diff = (at(1e-4) - at(-1e-4)) / 2e-4
        want = float(np.sum(grad[0].reshape(step.shape) * step))
        assert abs(diff - want) <= 1e-5 * max(1.0, abs(want)), (i, diff, want)


def test_reference_states_against_oracle():
    """The reference's forward pass is the oracle's: with o's gradient equal to a unit
    vector, dq is the column of the state that the oracle's o is a product with."""
    import oracle
    cfg = W.variant("tiny_fp32", T=5, H=1, h0=True)
    inp = W.make_inputs(cfg, 3)
    do = np.zeros_like(inp.q)
    do[..., 17] = 1.0
    dq = rule_bwd(inp.q, inp.k, inp.v, inp.g, inp.beta, do, inp.seq_bounds(), inp.h0)[0]
    o, _ = oracle.kda_ref_fwd(inp.q, inp.k, inp.v, inp.g, inp.beta, h0=inp.h0)
    assert np.allclose((dq * inp.q).sum(-1), o[..., 17], rtol=1e-12, atol=1e-12)


def test_refusals():
    import gated_delta_rule_63_amd as kda
    L = kda.lib()

    def d(B=1, T=64, H=2, K=128, N=None, dt=0, ws=None):
        need = 1 << 40 if ws is None else ws
        return kda.Desc(B, T, H, K, 128, B if N is None else N, dt, 1, P if need else None, need)

    def call(desc, fn="kda_bwd", cu=None, **kw):
        a = dict(zip("q k v g beta cu h0 do dhT dq dk dv dg db dh0".split(), [P] * 15))
        a.update(cu=cu, **kw)
        return getattr(L, fn)(*a.values(), ctypes.byref(desc) if desc else None, None)

    for fn in ("kda_bwd", "kda_gdn_bwd"):
        assert call(None, fn) == -1
        assert call(d(K=64), fn) == -3 and call(d(dt=7), fn) == -4
        assert call(d(N=3), fn) == -2 and call(d(B=2, N=3), fn, cu=P) == -2
        for name in ("q", "k", "v", "g", "beta", "do", "dq", "dk", "dv", "dg", "db"):
            assert call(d(), fn, **{name: None}) == -1, name
        assert call(d(), fn, do=ctypes.c_void_p(0x10004)) == -3          # not 16-byte aligned
        for name in ("q", "k", "v", "dq", "dk", "dv"):
            assert call(d(), fn, **{name: ctypes.c_void_p(0x10008)}) == -3, name
        x = d()
        x.workspace = 0x10008
        assert call(x, fn) == -3
        assert call(d(H=1 << 17, T=1), fn) == -2 and call(d(B=1 << 13, T=1, H=1 << 10, N=1 << 13), fn) == -2
        assert call(d(ws=0), fn) == -5 and call(d(ws=4 * 221824 - 1), fn) == -5
        assert call(d(B=1 << 12, T=1 << 16, H=64, N=1 << 12), fn) == -2  # 2^29 chunks
        assert call(d(B=1 << 6, T=0, H=1 << 15), fn) == -2               # 2^21 chains without a chunk
    # two chunks of two heads; with B == N == 1 the packed use may need one slot more
    size = lambda x: L.kda_bwd_workspace_size(ctypes.byref(x))
    assert size(d()) == 3 * 2 * 221824 and size(d(B=2, T=33)) == 4 * 2 * 221824
    assert size(d(N=5)) == 7 * 2 * 221824 and size(d(K=64)) == 0
    assert L.kda_bwd_workspace_size(None) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    from gated_delta_rule_63_amd import _ops
    z = lambda *s, **k: torch.zeros(*s, **k)
    q, g, b = z(2, 5, 3, 128), z(2, 5, 3, 128), z(2, 5, 3)
    st = z(2, 3, 128, 128)
    chk = lambda *a, s=False: _ops._check_bwd(*a, s, _device=False)
    chk(q, q, q, g, b, q, None, st, st)
    chk(q, q, q, z(2, 5, 3), b, q, None, None, None, s=True)
    for bad in [(q, q, q, g, b, q.bfloat16(), None, st, st), (q, q, q, g, b, z(2, 5, 128, 3).transpose(2, 3), None, st, st),
                (q, q, q, g, b, z(2, 4, 3, 128), None, st, st), (q, q, q, g, b, q, None, z(1, 3, 128, 128), st),
                (q, q, q, g, b, q, None, st, st.double()), (q, q, q, z(2, 5, 3), b, q, None, st, st)]:
        with pytest.raises(ValueError):
            chk(*bad)


# ------------------------------------------------------------------------- GPU

@pytest.fixture
def torch_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _grads(inp, seed, dhT=True):
    rng = np.random.default_rng(seed)
    do = rng.standard_normal(inp.q.shape, dtype=np.float32)
    c = inp.cfg
    return do, (0.1 * rng.standard_normal((c.N, c.H, 128, 128), dtype=np.float32) if dhT else None)


def _run(torch, inp, do, dhT, scalar=False, **kw):
    import gated_delta_rule_63_amd as kda
    from gpu_util import to_device
    t = to_device(inp, inp.cfg.dtype)
    dev = lambda x: None if x is None else torch.from_numpy(x).cuda()
    g = dev(inp.g_scalar()) if scalar else t["g"]
    f = kda.gdn_bwd if scalar else kda.bwd
    return f(t["q"], t["k"], t["v"], g, t["beta"], dev(do), cu_seqlens=t["cu"], initial_state=t["h0"],
             d_final_state=dev(dhT), **kw)


def _check(got, ref, inp, what):
    half = 2.0 ** -8 if inp.cfg.dtype == "bf16" else 0.0
    names = ["dq", "dk", "dv", "dg", "dbeta", "dh0"]
    x = {n: y.float().cpu().numpy() for n, y in zip(names, got)}
    r = dict(zip(names, ref))
    for n in names:
        scale = None
        if n == "dg":
            # a sum over up to 32 tokens of differences of the terms q dq and k dk:
            # its rounding follows their size, which may be far above the sum's
            scale = max(W.rms(r["dg"]), W.rms(inp.q * r["dq"]) + W.rms(inp.k * r["dk"]))
            scale *= 128 ** 0.5 if r["dg"].ndim == 3 else 1.0
        within(x[n], r[n], f"{what} {n}", half if n in ("dq", "dk", "dv") else 0.0, scale)


CASES = [
    (W.variant("tiny_fp32", T=1, h0=True), False),
    (W.variant("tiny_fp32", T=31), False),
    (W.variant("tiny_fp32", B=3, T=33, H=3, h0=True), True),
    (W.variant("T8192_H96", T=1 + 31 + 32 + 33 + 70 + 17, H=3, seq_lens=(0, 1, 31, 0, 32, 33, 70, 17, 0), h0=True), True),
    (W.variant("T8192_H96", B=2, T=100, H=5), True),
    (W.variant("tiny_fp32", T=200, H=2, gate="zero", beta="one", h0=True), True),
    (W.variant("tiny_fp32", T=64, H=2, gate="floor", h0=True), True),
    (W.variant("tiny_fp32", T=90, H=2, gate="mild", keys="same", h0=True), True),
    (W.variant("tiny_fp32", T=65, H=2, gate="mild", keys="onehot"), False),
    (W.variant("tiny_fp32", T=40, H=2, beta="zero", h0=True), True),
    (W.variant("T8192_H96", T=515, H=17, gate="mild"), False),
    # above 32 (sequence, head) pairs the walks take 32 columns of V at a time
    (W.variant("T8192_H96", T=98, H=24, seq_lens=(0, 33, 1, 64), h0=True), True),
    (W.variant("tiny_fp32", B=3, T=35, H=20, gate="mild", h0=True), True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("cfg,dhT", CASES, ids=lambda c: getattr(c, "name", str(c)))
def test_bwd(torch_gpu, cfg, dhT):
    inp = W.make_inputs(cfg, 5)
    do, dh = _grads(inp, 6, dhT)
    got = _run(torch_gpu, inp, do, dh)
    ref = rule_bwd(inp.q, inp.k, inp.v, inp.g, inp.beta, do, inp.seq_bounds(), inp.h0, dh)
    _check(got, ref, inp, cfg.name)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [
    W.variant("tiny_fp32", B=2, T=67, H=3, gate="scalar", h0=True),
    W.variant("T8192_H96", T=130, H=2, seq_lens=(64, 1, 0, 65), gate="scalar_mild", h0=True),
    W.variant("T8192_H96", T=71, H=20, seq_lens=(40, 31), gate="scalar", h0=True),
], ids=lambda c: c.name)
def test_gdn_bwd(torch_gpu, cfg):
    inp = W.make_inputs(cfg, 8)
    do, dh = _grads(inp, 9)
    got = _run(torch_gpu, inp, do, dh, scalar=True)
    ref = rule_bwd(inp.q, inp.k, inp.v, inp.g_scalar(), inp.beta, do, inp.seq_bounds(), inp.h0, dh)
    _check(got, ref, inp, cfg.name)


@pytest.mark.gpu
@pytest.mark.parametrize("cfg", [W.CONFIGS["T8192_H96"], W.CONFIGS["varlen6_T8192_H96"]], ids=lambda c: c.name)
def test_bwd_full_size(torch_gpu, cfg):
    """The full workloads, two heads of them against the reference (heads do not mix)."""
    inp = W.make_inputs(cfg, 0)
    do, dh = _grads(inp, 1)
    got = _run(torch_gpu, inp, do, dh)
    h = [0, 95]
    cut = lambda x: np.ascontiguousarray(x[:, :, h])
    st = lambda x: None if x is None else np.ascontiguousarray(x[:, h])
    ref = rule_bwd(cut(inp.q), cut(inp.k), cut(inp.v), cut(inp.g), cut(inp.beta), cut(do), inp.seq_bounds(),
                   st(inp.h0), st(dh))
    part = W.Inputs(cfg, cut(inp.q), cut(inp.k), cut(inp.v), cut(inp.g), cut(inp.beta), None, None)
    _check([x[:, :, h] for x in got[:5]] + [got[5][:, h]], ref, part, cfg.name)


@pytest.mark.gpu
def test_bwd_is_deterministic_and_streams(torch_gpu):
    """Bitwise the same: again, with a caller's workspace full of NaN, on another stream,
    two calls at once on two streams."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    inp = W.make_inputs(W.variant("T8192_H96", T=300, H=7, seq_lens=(100, 0, 37, 163), h0=True), 2)
    do, dh = _grads(inp, 3)
    first = _run(torch, inp, do, dh)
    from gpu_util import to_device
    t = to_device(inp, "bf16")
    need = kda.bwd_workspace_size(t["q"], t["cu"])
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [_run(torch, inp, do, dh, workspace=ws)]
    torch.cuda.synchronize()
    got += [_run(torch, inp, do, dh, stream=s) for s in (s1, s2)]
    torch.cuda.synchronize()
    for other in got:
        assert all(torch.equal(x, y) for x, y in zip(first, other))


@pytest.mark.gpu
def test_bwd_in_a_graph(torch_gpu):
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    from gpu_util import to_device
    inp = W.make_inputs(W.variant("T8192_H96", T=200, H=4, h0=True), 2)
    do, _ = _grads(inp, 3)
    t, d = to_device(inp, "bf16"), torch.from_numpy(do).cuda()
    run = lambda: kda.bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], d, initial_state=t["h0"])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for rep in range(3):
        d.copy_(torch.from_numpy(do).cuda() * (rep + 1))
        for x in out:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), rep


@pytest.mark.gpu
def test_bwd_leaves_other_rows(torch_gpu):
    """Tokens behind the last sequence are neither read into anything nor written; dh0
    may take dhT's place."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    from gpu_util import to_device
    cfg = W.variant("tiny_fp32", T=70, H=2, seq_lens=(30, 40), h0=True)
    inp = W.make_inputs(cfg, 4)
    do, dh = _grads(inp, 5)
    t = to_device(inp, "fp32")
    pad = lambda x: torch.cat([x, torch.full_like(x[:, :9], float("nan"))], 1).contiguous()
    q, k, v, g, b = (pad(t[n]) for n in ("q", "k", "v", "g", "beta"))
    d = pad(torch.from_numpy(do).cuda())
    outs = [torch.full_like(x, 7.0) for x in (q, k, v, g, b)]
    state = torch.from_numpy(dh).cuda()
    desc = kda.Desc(1, 79, 2, 128, 128, 2, 1, 1, None, 0)
    need = kda.lib().kda_bwd_workspace_size(ctypes.byref(desc))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    desc.workspace, desc.workspace_bytes = ws.data_ptr(), need
    ptr = lambda x: ctypes.c_void_p(x.data_ptr())
    rc = kda.lib().kda_bwd(*map(ptr, (q, k, v, g, b, t["cu"], t["h0"], d, state)), *map(ptr, outs), ptr(state),
                           ctypes.byref(desc), None)
    torch.cuda.synchronize()
    assert rc == 0
    assert all(bool((x[:, 70:] == 7.0).all()) for x in outs)
    ref = rule_bwd(inp.q, inp.k, inp.v, inp.g, inp.beta, do, inp.seq_bounds(), inp.h0, dh)
    _check([x[:, :70] for x in outs] + [state], ref, inp, "padded")


@pytest.mark.gpu
def test_bwd_far_elements(torch_gpu):
    """Elements of the tensors and of the workspace beyond 2^31: the last heads of a
    long, wide call are those of a call on them alone."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    T, H, m = 140000, 121, 40          # m alone: still 32 columns of V a workgroup
    assert T * H * 128 > 2 ** 31
    if torch.cuda.get_device_properties(0).total_memory < 230 << 30:
        pytest.skip("needs 170 GB of device memory")
    torch.cuda.empty_cache()
    gen = torch.Generator(device="cuda").manual_seed(2)

    def wide(dtype, scale, *s):
        x = torch.zeros(1, T, H, *s, dtype=dtype, device="cuda")
        x[:, :, -m:] = (torch.randn(1, T, m, *s, generator=gen, device="cuda") * scale).to(dtype)
        return x
    k, v, do = wide(torch.bfloat16, 128 ** -0.5, 128), wide(torch.bfloat16, 1.0, 128), wide(torch.float32, 1.0, 128)
    g, b = wide(torch.float32, 0.5, 128).abs_().neg_(), wide(torch.float32, 1.0).sigmoid_()
    args = (v, k, v, g, b, do)
    got = [x[:, :, -m:].clone() if x.dim() < 4 or x.shape[1] == T else x[:, -m:].clone() for x in kda.bwd(*args)]
    args = [x[:, :, -m:].contiguous() for x in args]
    want = kda.bwd(*args)
    assert all(bool(torch.isfinite(x).all()) and torch.equal(x, y) for x, y in zip(got, want))
    del k, v, do, g, b, args, got, want
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_bwd_without_tokens(torch_gpu):
    """T = 0: empty gradients, and the state's passes through."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    e = lambda *s: torch.zeros(*s, device="cuda")
    q, b, dh = e(2, 0, 3, 128), e(2, 0, 3), torch.randn(2, 3, 128, 128, device="cuda")
    got = kda.bwd(q, q, q, q, b, q, initial_state=dh, d_final_state=dh)
    assert all(x.numel() == 0 for x in got[:5]) and torch.equal(got[5], dh)
    got = kda.gdn_bwd(q, q, q, b, b, q)
    assert not bool(got[5].any())


@pytest.mark.gpu
def test_bwd_in_segments(torch_gpu):
    """A sequence's gradient in two calls, the second segment's state gradient handed to
    the first, is the gradient in one. The state between them comes from recurrent(),
    fp32 throughout; both ways are held to 1e-4 of the RMS each."""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    from gpu_util import to_device
    inp = W.make_inputs(W.variant("tiny_fp32", T=2500, H=3, gate="mild", h0=True), 9)
    do, dh = (torch.from_numpy(x).cuda() for x in _grads(inp, 10))
    t = to_device(inp, "fp32")
    x = [t[n] for n in ("q", "k", "v", "g", "beta")] + [do]
    whole = kda.bwd(*x, initial_state=t["h0"], d_final_state=dh)
    cut = 1111
    one, two = [u[:, :cut].contiguous() for u in x], [u[:, cut:].contiguous() for u in x]
    mid = t["h0"].clone()
    kda.recurrent(*one[:5], mid)
    b = kda.bwd(*two, initial_state=mid, d_final_state=dh)
    a = kda.bwd(*one, initial_state=t["h0"], d_final_state=b[5])
    for name, w, u, v in zip("dq dk dv dg dbeta".split(), whole, a, b):
        within(torch.cat([u, v], 1).cpu().numpy(), w.cpu().numpy(), name, tol=2e-4)
    within(a[5].cpu().numpy(), whole[5].cpu().numpy(), "dh0", tol=2e-4)


# ---- the fp32 gradients' own accuracy, measured on their own size

def _rms_off(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape and np.all(np.isfinite(got))
    return W.rms(got - ref) / W.rms(ref)


# RMS of the error over RMS of the result. A sum of 128 products rounds by 2^-24
# sqrt(128) = 7e-7 of itself, ten in a row by 2.2e-6. A decay's exponent, up to 58 for
# gates of -5, is a sum of up to eight gates, each partial sum rounded by at most
# 2^-19 ln 2 = 1.3e-6, 0.8e-6 RMS: 2e-6 together. 3e-6 of both; a factor of 3 for the
# terms of a sum over 16 tokens that exceed it.
RMS_BAR = 1e-5


def _check_rms(got, ref, what, bar=RMS_BAR):
    for n, i in (("dg", 3), ("dbeta", 4), ("dh0", 5)):
        off = _rms_off(got[i].cpu().numpy(), ref[i])
        print(f"{what} {n}: rms {off:.2e}", flush=True)
        assert off <= bar, f"{what} {n}: rms off by {off:.2e} (bar {bar:.0e})"


@pytest.mark.gpu
@pytest.mark.parametrize("cfg,scalar", [
    (W.variant("tiny_fp32", T=64, H=2, gate="floor", h0=True), False),
    (W.variant("tiny_fp32", T=64, H=2, gate="floor"), False),
    (W.variant("T8192_H96", T=131, H=3, gate="floor", seq_lens=(33, 2, 96), h0=True), False),
    (W.variant("T8192_H96", T=70, H=40, gate="floor"), False),
    (W.variant("tiny_fp32", T=64, H=2, gate="floor", h0=True), True),
    (W.variant("T8192_H96", T=131, H=3, gate="floor", seq_lens=(33, 2, 96)), True),
    (W.variant("tiny_fp32", T=100, H=2, h0=True), False),
    (W.variant("tiny_fp32", T=100, H=2, gate="scalar", h0=True), True),
    (W.variant("tiny_fp32", T=2500, H=1, gate="mild", h0=True), False),
    (W.variant("tiny_fp32", T=700, H=1, gate="scalar_mild", h0=True), True),
], ids=lambda c: getattr(c, "name", str(c)))
def test_bwd_fp32_gradients(torch_gpu, cfg, scalar):
    """dg, dbeta and dh0 on their own size, also where every gate is at its floor: dg
    then is e^-5 of the products q dq and k dk that it is a difference of."""
    inp = W.make_inputs(cfg, 12)
    do, dh = _grads(inp, 13)
    got = _run(torch_gpu, inp, do, dh, scalar=scalar)
    ref = rule_bwd(inp.q, inp.k, inp.v, inp.g_scalar() if scalar else inp.g, inp.beta, do, inp.seq_bounds(), inp.h0, dh)
    _check_rms(got, ref, cfg.name)
    within(got[3].cpu().numpy(), ref[3], f"{cfg.name} dg")     # no element off by 1e-4 of the RMS


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
def test_bwd_gate_of_a_zero_state(torch_gpu, scalar):
    """A token that starts from nothing has no gate gradient: exactly zero, and not what
    is left of two equal terms."""
    inp = W.make_inputs(W.variant("tiny_fp32", B=5, T=1, H=3, gate="scalar"), 14)
    do, dh = _grads(inp, 15)
    got = _run(torch_gpu, inp, do, dh, scalar=scalar)
    assert bool(got[0].any()) and not bool(got[3].any())


@pytest.mark.gpu
@pytest.mark.parametrize("scalar", [False, True])
@pytest.mark.parametrize("low,high", [(-5.5, -5.5), (-6.0, -6.0), (-8.0, -8.0), (-8.0, 0.0), (-16.0, 0.0)])
def test_bwd_stronger_gates(torch_gpu, scalar, low, high):
    """Gates below kda_fwd's range: down to -8 throughout, and lower where they are rare
    (-16 among gates of -0.1, one token in eight).
    Exponents reach 92, whose partial sums round by 2^-18 ln 2 = 2.6e-6 instead of 1.3e-6:
    twice RMS_BAR and, for single elements of dg, twice the bar of 1e-4."""
    inp = W.make_inputs(W.variant("tiny_fp32", T=101, H=2, gate="scalar" if scalar else "bj", h0=True), 16)
    rng = np.random.default_rng(17)
    g = rng.uniform(low, high, inp.g.shape).astype(np.float32)
    if low == -16.0:
        g = np.where(np.arange(101)[:, None, None] % 8 == 5, np.float32(-16.0), np.float32(-0.1)) * np.ones_like(g)
    inp.g[:] = g[..., :1] if scalar else g
    do, dh = _grads(inp, 18)
    got = _run(torch_gpu, inp, do, dh, scalar=scalar)
    ref = rule_bwd(inp.q, inp.k, inp.v, inp.g_scalar() if scalar else inp.g, inp.beta, do, inp.seq_bounds(), inp.h0, dh)
    for n, x, r in zip("dq dk dv".split(), got, ref):
        within(x.cpu().numpy(), r, n)
    _check_rms(got, ref, f"[{low}, {high}]", 2 * RMS_BAR)
    within(got[3].cpu().numpy(), ref[3], "dg", tol=2e-4)


@pytest.mark.gpu
def test_bwd_two_calls_at_once(torch_gpu):
    """Calls that run at the same time on two streams, on the same inputs and each with a
    gradient of its own, give what each gives alone: their workspaces are apart. (On long
    sequences with few heads, so that one does not fill the chip.)"""
    torch = torch_gpu
    import gated_delta_rule_63_amd as kda
    from gpu_util import to_device
    inp = W.make_inputs(W.variant("T8192_H96", T=4096, H=4, h0=True), 19)
    t = to_device(inp, "bf16")
    do = [torch.from_numpy(_grads(inp, seed, False)[0]).cuda() for seed in (20, 21)]
    run = lambda d, **kw: kda.bwd(t["q"], t["k"], t["v"], t["g"], t["beta"], d, initial_state=t["h0"], **kw)
    alone = [run(d) for d in do]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [run(d, stream=s) for _ in range(3) for d, s in zip(do, streams)]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(out, alone[i % 2])), i
    assert not torch.equal(alone[0][0], alone[1][0])

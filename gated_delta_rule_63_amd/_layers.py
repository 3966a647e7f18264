"""Torch marshalling of the rule with a vector state, of the residual's addition with a
norm between two layers, and of a step of beam search (include/kda.h). Outputs and
workspaces are allocated on the call's stream; nothing is recorded by torch.autograd (see
_ops)."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._lib import KDA_F32, BeamDesc, NormDesc, ScanDesc, lib
from ._ops import _DTYPES, _Tensor, _call, _on, _ptr, _rows

SCAN_CHUNK = 128


def _plain(name, t, shape, dtype, device, _device=True):
    """A tensor the kernels read or write: contiguous, of this shape (a torch.Size), type and device."""
    if t is not None:
        _rows(name, t, shape, dtype, device, _device)


_MOST = 0x7fffffff                    # of the descriptors' 32-bit fields: ctypes would cut off silently


def _fits(*n):
    if max(n) > _MOST:
        raise ValueError("a dimension is beyond 32 bits")


def _bytes(n: int, like: torch.Tensor) -> _Tensor:
    return like.new_empty(n, dtype=torch.uint8) if n else None


def _with(desc, ws: _Tensor):
    if ws is not None:
        desc.workspace, desc.workspace_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    return ctypes.byref(desc)


# ------------------------------------------------------- the rule with a vector state

def _scan_desc(x, cu_seqlens, leaky=False) -> ScanDesc:
    shape = x.shape
    N = shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
    C = shape[2] if len(shape) == 3 else shape[2:].numel()
    if not 0 < x.numel() <= _MOST or N > _MOST:       # (no dimension is larger than all elements, if there are any)
        _fits(shape[0], shape[1], C, N)
    return ScanDesc(shape[0], shape[1], C, N, _DTYPES[x.dtype], leaky, None, 0)


def _scan_state(d: ScanDesc, x) -> torch.Size:
    return torch.Size((d.num_seqs, *x.shape[2:]))


def _check_scan(x, g, cu_seqlens, leaky=False, _device=True) -> ScanDesc:
    shape, device = x.shape, x.device
    if len(shape) < 3 or x.dtype not in _DTYPES:
        raise ValueError("x must be a bfloat16 or float32 [B, T, ...] tensor")
    _rows("x", x, shape, x.dtype, device, _device)
    _rows("g", g, shape, torch.float32, device, False)
    if cu_seqlens is not None:
        if (cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1
                or not cu_seqlens.is_contiguous() or cu_seqlens.device != device):
            raise ValueError("cu_seqlens must be a contiguous int32 [N + 1] tensor on x's device")
        if shape[0] != 1:
            raise ValueError("with cu_seqlens the batch dimension must be 1 (sequences packed into one row)")
    return _scan_desc(x, cu_seqlens, leaky)


def _states_shape(d: ScanDesc, x, cu_seqlens):
    """Shape of the states at chunk starts: [B, ceil(T / 128), ...], packed [1, T // 128 + N, ...]."""
    if cu_seqlens is None:
        return torch.Size((d.B, (d.T + SCAN_CHUNK - 1) // SCAN_CHUNK, *x.shape[2:]))
    return torch.Size((1, d.T // SCAN_CHUNK + d.num_seqs, *x.shape[2:]))


def _workspace(given: _Tensor, need: int, like: torch.Tensor) -> _Tensor:
    if given is None:
        return _bytes(need, like)
    if given.device != like.device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the first argument's device")
    return given


def scan_workspace_size(x: torch.Tensor, cu_seqlens: _Tensor = None) -> int:
    """Bytes of device workspace scan() uses for inputs shaped like x (0 for most shapes)."""
    return int(lib().kda_scan_workspace_size(ctypes.byref(_scan_desc(x, cu_seqlens))))


def scan(x: torch.Tensor, g: torch.Tensor, cu_seqlens: _Tensor = None, initial_state: _Tensor = None, leaky: bool = False,
         output_chunk_states: bool = False, out: _Tensor = None, final_state: _Tensor = None,
         stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[_Tensor, ...]:
    """The rule with a vector state, channel by channel: h_t = exp(g_t) h_{t-1} + x_t, or
    leaky: h_t = exp(g_t) h_{t-1} + (1 - exp(g_t)) x_t. x [B, T, ...] bf16 or fp32 with
    any trailing dimensions (a heads' and a channels', or one); g fp32, of x's shape: a
    log-decay, -inf for a reset. cu_seqlens int32 [N + 1]: sequences packed into one row,
    as for fwd(). initial_state fp32 [N, ...].

    Returns (y, final_state, chunk_states): every token's state in x's dtype, the last ones
    in fp32, and with output_chunk_states the states that enter each chunk of 128 tokens,
    which scan_bwd() takes ([B, ceil(T / 128), ...]; packed [1, T // 128 + N, ...], where
    sequence n's begin at row cu[n] // 128 + n and rows without a chunk are unset), else
    None. Rows of y of tokens that belong to no sequence are left as they were: unset without
    out. Gates above 0 make a state grow: gates of 16 tokens in a row, or fewer, sum to 88 at
    most where the state is not zero, and longer runs to anything that leaves every state
    finite. out may be x, final_state initial_state. workspace: an optional device tensor of
    scan_workspace_size() bytes, used by one call at a time; allocated otherwise."""
    d = _check_scan(x, g, cu_seqlens, leaky)
    state = _scan_state(d, x)
    _plain("initial_state", initial_state, state, torch.float32, x.device)
    _plain("final_state", final_state, state, torch.float32, x.device)
    _plain("out", out, x.shape, x.dtype, x.device)
    with _on(x.device, stream) as s:
        y = torch.empty_like(x) if out is None else out
        hT = g.new_empty(state) if final_state is None else final_state
        kept = g.new_empty(_states_shape(d, x, cu_seqlens)) if output_chunk_states else None
        ws = _workspace(workspace, int(lib().kda_scan_workspace_size(ctypes.byref(d))), x)
        _call("kda_scan", _ptr(x), _ptr(g), _ptr(cu_seqlens), _ptr(initial_state), _ptr(y), _ptr(hT), _ptr(kept),
              _with(d, ws), s)
    return y, hT, kept


def scan_bwd(x: torch.Tensor, g: torch.Tensor, dy: torch.Tensor, cu_seqlens: _Tensor = None, initial_state: _Tensor = None,
             d_final_state: _Tensor = None, chunk_states: _Tensor = None, leaky: bool = False,
             stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of scan(). The first two arguments, cu_seqlens and initial_state are the
    forward's; dy (x's dtype) and d_final_state (fp32, None: zero) the gradients with
    respect to its outputs; chunk_states what the forward returned (None: formed again, at
    the cost of reading x and g once more). Returns (dx, dg, d_initial_state), dx in x's
    dtype, the others fp32. Rows of tokens that belong to no sequence are unset. workspace:
    an optional device tensor of scan_bwd_workspace_size() bytes, used by one call at a
    time; allocated otherwise."""
    d = _check_scan_bwd(x, g, dy, cu_seqlens, initial_state, d_final_state, chunk_states, leaky)
    with _on(x.device, stream) as s:
        dx, dg = torch.empty_like(x), torch.empty_like(g)
        dh0 = g.new_empty(_scan_state(d, x))
        need = int(lib().kda_scan_bwd_workspace_size(ctypes.byref(d), chunk_states is not None))
        ws = _workspace(workspace, need, x)
        _call("kda_scan_bwd", _ptr(x), _ptr(g), _ptr(cu_seqlens), _ptr(initial_state), _ptr(chunk_states), _ptr(dy),
              _ptr(d_final_state), _ptr(dx), _ptr(dg), _ptr(dh0), _with(d, ws), s)
    return dx, dg, dh0


def _check_scan_bwd(x, g, dy, cu_seqlens, initial_state, d_final_state, chunk_states, leaky=False, _device=True) -> ScanDesc:
    d = _check_scan(x, g, cu_seqlens, leaky, _device)
    state = _scan_state(d, x)
    _plain("dy", dy, x.shape, x.dtype, x.device, _device)
    _plain("initial_state", initial_state, state, torch.float32, x.device, _device)
    _plain("d_final_state", d_final_state, state, torch.float32, x.device, _device)
    _plain("chunk_states", chunk_states, _states_shape(d, x, cu_seqlens), torch.float32, x.device, _device)
    return d


def scan_bwd_workspace_size(x: torch.Tensor, cu_seqlens: _Tensor = None, with_states: bool = True) -> int:
    """Bytes of device workspace scan_bwd() uses for inputs shaped like x, with chunk_states or without."""
    return int(lib().kda_scan_bwd_workspace_size(ctypes.byref(_scan_desc(x, cu_seqlens)), with_states))


def scan_recurrent(x: torch.Tensor, g: torch.Tensor, pool: torch.Tensor, slots: _Tensor = None, out_slots: _Tensor = None,
                   cu_seqlens: _Tensor = None, leaky: bool = False, out: _Tensor = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """scan() token by token for a few tokens per sequence, on states in a pool ([P, ...], fp32 or
    bf16), which is updated in place; slots, out_slots and empty places as for recurrent().
    Returns y in x's dtype; out may be x."""
    d = _check_scan_recurrent(x, g, pool, slots, out_slots, cu_seqlens, out, leaky)
    with _on(x.device, stream) as s:
        y = torch.empty_like(x) if out is None else out
        _call("kda_scan_recurrent", _ptr(x), _ptr(g), _ptr(cu_seqlens), _ptr(slots), _ptr(out_slots), _ptr(pool),
              pool.shape[0], _DTYPES[pool.dtype], _ptr(y), ctypes.byref(d), s)
    return y


def _check_scan_recurrent(x, g, pool, slots, out_slots, cu_seqlens, out, leaky=False, _device=True) -> ScanDesc:
    d = _check_scan(x, g, cu_seqlens, leaky, _device)
    device, shape = x.device, pool.shape
    if shape[1:] != x.shape[2:] or not pool.is_contiguous() or pool.dtype not in _DTYPES or pool.device != device:
        raise ValueError(f"pool must be a contiguous float32 or bfloat16 [P, {', '.join(map(str, x.shape[2:]))}] tensor on x's device")
    if shape[0] > _MOST:
        _fits(shape[0])
    if slots is None and shape[0] < d.num_seqs:
        raise ValueError("pool has fewer slots than there are sequences")
    for name, t, n in (("slots", slots, d.num_seqs), ("out_slots", out_slots, d.B * d.T)):
        if t is not None and (t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or t.device != device):
            raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements on x's device")
    _plain("out", out, x.shape, x.dtype, x.device, _device)
    return d


# ------------------------------------------------------- the residual's addition and a norm

def _check_norm(x, residual, weight, _device=True) -> NormDesc:
    shape, device, dtype = x.shape, x.device, x.dtype
    if len(shape) < 1 or shape[-1] < 1 or dtype not in _DTYPES:
        raise ValueError("x must be a bfloat16 or float32 [..., C] tensor")
    C, res = shape[-1], dtype
    _rows("x", x, shape, dtype, device, _device)
    _rows("weight", weight, shape[-1:], torch.float32, device, False)
    if residual is not None:
        res = residual.dtype
        if res != dtype and res != torch.float32:
            raise ValueError("residual must have x's dtype or be float32")
        _rows("residual", residual, shape, res, device, False)
    if C > _MOST:
        _fits(C)
    return NormDesc(x.numel() // C, C, _DTYPES[dtype], _DTYPES[res], None, 0)


def add_norm(x: torch.Tensor, residual: _Tensor, weight: torch.Tensor, eps: float = 1e-5, out: _Tensor = None,
             residual_out: _Tensor = None, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """r = x + residual, and the RMS norm of r over the last dimension, r / sqrt(mean(r^2) + eps) *
    weight. x [..., C] bf16 or fp32; residual of the same shape, in x's dtype or fp32, or None
    (r is x then); weight fp32 [C]. Returns (y in x's dtype, r in residual's). out may be x,
    residual_out may be residual (the stream updated in place). With out in x's place and no
    residual r is overwritten, and returned as None: add_norm_bwd() needs a copy of x then."""
    d = _check_norm(x, residual, weight)
    _check_norm_out(x, residual, weight, out, residual_out)
    with _on(x.device, stream) as s:
        y = torch.empty_like(x) if out is None else out
        r = _sum_out(x, residual, residual_out)
        if residual is None and out is not None and out.data_ptr() == x.data_ptr():
            r = None
        _call("kda_add_norm", _ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(y), _ptr(r) if residual is not None else None,
              ctypes.byref(d), s)
    return y, r


def _check_norm_out(x, residual, weight, out, residual_out, _device=True):
    """Outputs may lie exactly where x or residual does, and are apart from all else. (Straight on, since a
    small call's time is the host's: 1.6 us in place, 4.1 with tensors of their own.)"""
    if out is None and residual_out is None:
        return
    n, px, pw, m = x.nbytes, x.data_ptr(), weight.data_ptr(), 4 * x.shape[-1]
    pr = nr = po = 0
    if residual is not None:
        pr, nr = residual.data_ptr(), n if residual.dtype == x.dtype else 2 * n
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is not None:
        po = px
        if out is not x:
            _rows("out", out, x.shape, x.dtype, x.device, _device)
            po = out.data_ptr()
        if -n < po - px < n and po != px or -n < po - pr < nr and (po != pr or n != nr) or -n < po - pw < m:
            raise ValueError("out overlaps an input and does not lie exactly in its place")
    if residual_out is not None:
        ps = pr
        if residual_out is not residual:
            _rows("residual_out", residual_out, residual.shape, residual.dtype, residual.device, _device)
            ps = residual_out.data_ptr()
        if -nr < ps - px < n and (ps != px or n != nr) or -nr < ps - pr < nr and ps != pr or -nr < ps - pw < m:
            raise ValueError("residual_out overlaps an input and does not lie exactly in its place")
        if out is not None and -n < po - ps < nr:
            raise ValueError("out and residual_out overlap")


def _sum_out(x, residual, residual_out):
    if residual is None:
        return x
    return torch.empty_like(residual) if residual_out is None else residual_out


def add_norm_q8(x: torch.Tensor, residual: _Tensor, weight: torch.Tensor, group: int = 0, eps: float = 1e-5,
                residual_out: _Tensor = None, stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """add_norm() with y in 8 bits: scale = max(amax |y|, 2^-40) / 448 over a row (group=0) or over
    each 128 channels (group=128, C a multiple of it), and y / scale rounded to
    float8_e4m3fn. Returns (q [..., C], scales fp32 [...] or [..., C / 128], r)."""
    d = _check_norm(x, residual, weight)
    if group not in (0, 128) or (group and d.C % group):
        raise ValueError("group must be 0 (a row) or 128, with a multiple of 128 channels")
    _check_norm_out(x, residual, weight, None, residual_out)
    with _on(x.device, stream) as s:
        q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        scales = weight.new_empty((*x.shape[:-1], d.C // group) if group else x.shape[:-1])
        r = _sum_out(x, residual, residual_out)
        _call("kda_add_norm_q8", _ptr(x), _ptr(residual), _ptr(weight), eps, group, _ptr(q), _ptr(scales),
              _ptr(r) if residual is not None else None, ctypes.byref(d), s)
    return q, scales, r


def add_norm_bwd(r: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor, dr: _Tensor = None, eps: float = 1e-5,
                 stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of add_norm(). r is the sum that it returned (x without a residual), dy the
    gradient with respect to y (bf16 or fp32; r in dy's dtype or fp32), dr (r's dtype, None:
    zero) that with respect to r from where else it is used. Returns (dx in dy's dtype,
    d_residual in r's, dweight fp32): the gradients of x and of residual are the same sum, and
    one tensor where the dtypes are. dweight takes every row. workspace: an optional device
    tensor of add_norm_bwd_workspace_size() bytes, used by one call at a time; allocated
    otherwise."""
    d = _check_norm_bwd(r, weight, dy, dr)
    with _on(r.device, stream) as s:
        dx, dw = torch.empty_like(dy), torch.empty_like(weight)
        dres = dx if r.dtype == dy.dtype else torch.empty_like(r)
        ws = _workspace(workspace, int(lib().kda_add_norm_bwd_workspace_size(ctypes.byref(d))), r)
        _call("kda_add_norm_bwd", _ptr(r), _ptr(weight), eps, _ptr(dy), _ptr(dr), _ptr(dx), None if dres is dx else _ptr(dres),
              _ptr(dw), _with(d, ws), s)
    return dx, dres, dw


def add_norm_bwd_workspace_size(dy: torch.Tensor) -> int:
    """Bytes of device workspace add_norm_bwd() uses for a gradient shaped like dy, on the current device."""
    if dy.dim() < 1 or dy.shape[-1] < 1:
        raise ValueError("dy must be a [..., C] tensor")
    C = dy.shape[-1]
    _fits(C)
    return int(lib().kda_add_norm_bwd_workspace_size(ctypes.byref(NormDesc(dy.numel() // C, C, KDA_F32, KDA_F32, None, 0))))


def _check_norm_bwd(r, weight, dy, dr, _device=True) -> NormDesc:
    if r is None:
        raise ValueError("r must be the sum that add_norm() normed")
    d = _check_norm(dy, r, weight, _device)
    _plain("dr", dr, r.shape, r.dtype, r.device, _device)
    return d


# ------------------------------------------------------- beam search

def _check_beam(logits, scores, k, done, eos, _device=True) -> BeamDesc:
    shape, device = logits.shape, logits.device
    if len(shape) != 3 or logits.dtype not in _DTYPES:
        raise ValueError("logits must be a bfloat16 or float32 [B, W, V] tensor")
    B, W, V = shape
    _rows("logits", logits, shape, logits.dtype, device, _device)
    _rows("scores", scores, shape[:2], torch.float32, device, False)
    if done is not None:
        if done.dtype not in (torch.bool, torch.uint8):
            raise ValueError("done must be a bool or uint8 [B, W] tensor")
        _rows("done", done, shape[:2], done.dtype, device, False)
        if not 0 <= eos < V:
            raise ValueError("with done, eos must be a token")
    k = W if k is None else k
    if not (1 <= W <= 64 and 1 <= k <= 64):
        raise ValueError("beams and k must be 1 to 64")
    if not 0 < logits.numel() <= _MOST:
        _fits(B, V)
    return BeamDesc(B, W, V, k, _DTYPES[logits.dtype], eos, None, 0)


def beam_select(logits: torch.Tensor, scores: torch.Tensor, k: Optional[int] = None, done: _Tensor = None, eos: int = -1,
                stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[torch.Tensor, ...]:
    """The k (None: W) best continuations of each batch entry's W beams: the largest of
    scores[b, w] + log_softmax(logits[b, w])[v] over beams and tokens, descending, ties to the
    lowest beam, then token. logits [B, W, V] bf16 or fp32, scores fp32 [B, W] (-inf: a dead
    beam). done: bool [B, W], beams that have ended: each has one candidate, eos with its score
    unchanged, and its logits are not read. Returns (scores fp32, parents int32, tokens int32),
    each [B, k]; places beyond the last candidate hold -inf, -1, -1. workspace: an optional device
    tensor of beam_workspace_size() bytes, used by one call at a time; allocated otherwise."""
    d = _check_beam(logits, scores, k, done, eos)
    with _on(logits.device, stream) as s:
        ws = _workspace(workspace, int(lib().kda_beam_workspace_size(ctypes.byref(d))), logits)
        best = scores.new_empty(d.B, d.K)
        parents = torch.empty_like(best, dtype=torch.int32)
        tokens = torch.empty_like(parents)
        _call("kda_beam_select", _ptr(logits), _ptr(scores), _ptr(done), _ptr(best), _ptr(parents), _ptr(tokens), _with(d, ws), s)
    return best, parents, tokens


def beam_workspace_size(logits: torch.Tensor, k: Optional[int] = None) -> int:
    """Bytes of device workspace beam_select() uses for logits shaped like these, on the current device."""
    if logits.dim() != 3:
        raise ValueError("logits must be [B, W, V]")
    B, W, V = logits.shape
    k = W if k is None else k
    _fits(B, W, V, k)
    d = BeamDesc(B, W, V, k, _DTYPES.get(logits.dtype, -1), -1, None, 0)
    return int(lib().kda_beam_workspace_size(ctypes.byref(d)))


def _check_reorder(pool, slots, parents, out, _device=True):
    if pool.dim() < 1 or not pool.is_contiguous() or (_device and not pool.is_cuda):
        raise ValueError("pool must be a contiguous device tensor [P, ...]")
    if slots.dim() != 2 or not 1 <= slots.shape[1] <= 64:
        raise ValueError("slots must be [B, W] with 1 to 64 beams")
    if pool.shape[0] > _MOST or slots.shape[0] > _MOST:
        _fits(pool.shape[0], slots.shape[0])
    for name, t in (("slots", slots), ("parents", parents), ("out", out)):
        _plain(name, t, slots.shape, torch.int32, pool.device, _device)
    if out is not None:
        n, at = out.nbytes, out.data_ptr()                # three tensors of one size
        if -n < at - slots.data_ptr() < n or -n < at - parents.data_ptr() < n:
            raise ValueError("out may not overlap slots or parents")


def beam_reorder(pool: torch.Tensor, slots: torch.Tensor, parents: torch.Tensor, out: _Tensor = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Reorders the states of a pool ([P, ...], of recurrent(), scan_recurrent() or any other) in
    place after a selection: slots int32 [B, W] names the slot of each beam, parents int32 [B, W]
    the beam that each new one continues. Returns the slots of the new beams: a beam's
    first child keeps its slot, further ones get copies in the slots of beams without children
    (the same slots in each entry, and the same result for every pool of a model). A parent
    outside [0, W) is an empty place: it gets a free slot, whose state is left as it is. out may
    not overlap slots or parents."""
    _check_reorder(pool, slots, parents, out)
    with _on(pool.device, stream) as s:
        new = torch.empty_like(slots) if out is None else out
        B, W = slots.shape
        _call("kda_beam_reorder", _ptr(pool), pool.shape[0], pool.shape[1:].numel() * pool.element_size(),
              _ptr(slots), _ptr(parents), _ptr(new), B, W, s)
    return new

"""Torch marshalling of the operators around the rule: its gradient, its recurrent
form over a pool of states, and what comes right before and after it
(include/kda.h). Outputs and workspaces are allocated on the call's stream.

Nothing here (nor fwd() and its kin) is recorded by torch.autograd: results do not
require gradients whatever the inputs do, and a model that trains through these calls
joins each with its gradient itself, in a torch.autograd.Function whose forward calls
the one and whose backward calls the other."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import D, _check_inputs, _check_out, _check_state, _desc
from ._lib import ACTIVATIONS, KDA_BF16, KDA_F32, Desc, KDAError, lib

_Tensor = Optional[torch.Tensor]
_DTYPES = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}


def _ptr(t: _Tensor) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _f32(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t, dtype=torch.float32)   # 1.2 us; torch.empty with shape and device 3.0


# the stream's handle without a torch.cuda.Stream around it: 0.1 us against 1.1
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


class _Here:
    """The call's stream where its device and stream are current already."""

    def __init__(self, raw):
        self.raw = raw

    def __enter__(self):
        return self.raw

    def __exit__(self, *_):
        pass


def _on(device: torch.device, stream: Optional[torch.cuda.Stream]):
    """Makes `device` and the call's stream current, so that launches and
    allocations go there; yields the stream as the C ABI takes it. (Entering torch's
    contexts costs more than a small kernel: where they would change nothing they are
    left out.)"""
    if stream is None and torch.cuda.current_device() == device.index:
        return _Here(_raw_stream(device.index))
    return _there(device, stream)


@contextlib.contextmanager
def _there(device, stream):
    with torch.cuda.device(device):
        s = stream or torch.cuda.current_stream(device)
        if s.device != device:
            raise ValueError("stream must belong to the tensors' device")
        with torch.cuda.stream(s):
            yield s.cuda_stream


def _call(entry: str, *args) -> None:
    rc = getattr(lib(), entry)(*args)
    if rc != 0:
        raise KDAError(rc, entry)


# ----------------------------------------------------------------- the gradient

def bwd_workspace_size(q: torch.Tensor, cu_seqlens: _Tensor = None) -> int:
    """Bytes of device workspace bwd() / gdn_bwd() use for inputs shaped like q."""
    return int(lib().kda_bwd_workspace_size(ctypes.byref(_desc(q, cu_seqlens))))


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, do: torch.Tensor,
        cu_seqlens: _Tensor = None, initial_state: _Tensor = None, d_final_state: _Tensor = None,
        stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of fwd(). The first arguments are the forward's; do (fp32 [B, T, H, 128],
    16-byte aligned) and d_final_state (fp32 [N, H, 128, 128]; None: zero) are the
    gradients with respect to its outputs. Returns (dq, dk, dv, dg, dbeta,
    d_initial_state): dq, dk, dv in q's dtype, the others fp32. Rows of tokens that
    belong to no sequence (cu_seqlens) are unset, as fwd()'s are: hand the first cu[N]
    tokens alone to block_out() and to the gradients of the block operators, whose sums
    take every row. Nothing is kept from the forward; states are recomputed.
    Gates may go down to -8; where eight tokens in a row have gates that sum to less
    than -87 the gradient may be NaN, without an error (fwd() ends earlier, at about
    -5.4 over 16 tokens). workspace: an optional uint8 device tensor of
    bwd_workspace_size() bytes, used by one call at a time; allocated otherwise."""
    return _bwd("kda_bwd", q, k, v, g, beta, do, cu_seqlens, initial_state, d_final_state, stream, workspace)


def gdn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, do: torch.Tensor,
            cu_seqlens: _Tensor = None, initial_state: _Tensor = None, d_final_state: _Tensor = None,
            stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of gdn_fwd(): as bwd(), with g and dg [B, T, H], and with its limit on
    the gates."""
    return _bwd("kda_gdn_bwd", q, k, v, g, beta, do, cu_seqlens, initial_state, d_final_state, stream, workspace)


def _check_bwd(q, k, v, g, beta, do, cu_seqlens, initial_state, d_final_state, scalar_gate, _device=True):
    _check_inputs(q, k, v, g, beta, cu_seqlens, scalar_gate=scalar_gate, _device=_device)
    d = _desc(q, cu_seqlens)
    sshape = (d.num_seqs, q.shape[2], D, D)
    _check_out("do", do, q.shape, q.device)
    _check_state("initial_state", initial_state, sshape, q.device)
    _check_state("d_final_state", d_final_state, sshape, q.device)
    return d, sshape


def _bwd(entry, q, k, v, g, beta, do, cu_seqlens, initial_state, d_final_state, stream, workspace):
    d, sshape = _check_bwd(q, k, v, g, beta, do, cu_seqlens, initial_state, d_final_state, entry == "kda_gdn_bwd")
    if workspace is not None and (workspace.device != q.device or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on q's device")
    with _on(q.device, stream) as s:
        if workspace is None:
            need = int(lib().kda_bwd_workspace_size(ctypes.byref(d)))
            workspace = q.new_empty(need, dtype=torch.uint8)
        d.workspace = workspace.data_ptr()
        d.workspace_bytes = workspace.numel() * workspace.element_size()
        outs = [torch.empty_like(x) for x in (q, k, v, g, beta)]
        dh0 = q.new_empty(sshape, dtype=torch.float32)
        _call(entry, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(initial_state), _ptr(do),
              _ptr(d_final_state), *map(_ptr, outs), _ptr(dh0), ctypes.byref(d), s)
    return (*outs, dh0)


# ------------------------------------------------- token by token over a state pool

def recurrent(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
              pool: torch.Tensor, slots: _Tensor = None, out_slots: _Tensor = None, cu_seqlens: _Tensor = None,
              out: _Tensor = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The rule token by token for a few tokens per sequence, on states in a pool
    ([P, H, 128, 128], fp32 or bf16), which is updated in place. q, k, v, g [B, T, H, 128],
    beta [B, T, H], cu_seqlens as for fwd(). slots: int32 [N], the slot that sequence n
    starts from (None: slot n); a value outside [0, P) is an empty place of the batch,
    whose rows of the output are left as they were (unset without `out`). out_slots:
    int32, one per token ([B, T]), where the state after that token goes (outside
    [0, P): not kept); None: the last state goes back to the sequence's slot. A slot
    that is written may not be used by another sequence of the call. Returns o, fp32
    [B, T, H, 128]."""
    return _recurrent("kda_recurrent", q, k, v, g, beta, pool, slots, out_slots, cu_seqlens, out, stream)


def gdn_recurrent(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
                  pool: torch.Tensor, slots: _Tensor = None, out_slots: _Tensor = None, cu_seqlens: _Tensor = None,
                  out: _Tensor = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """recurrent() with one gate per (token, head): g [B, T, H]. As q, k, v, pool and out, it
    has to start on a multiple of 16 bytes (a slice of tokens of one sequence with an odd
    number of heads may not: clone() it)."""
    return _recurrent("kda_gdn_recurrent", q, k, v, g, beta, pool, slots, out_slots, cu_seqlens, out, stream)


def _check_recurrent(q, k, v, g, beta, pool, slots, out_slots, cu_seqlens, out, scalar_gate, _device=True):
    _check_inputs(q, k, v, g, beta, cu_seqlens, scalar_gate=scalar_gate, _device=_device)
    d = _desc(q, cu_seqlens)
    if (pool.dim() != 4 or tuple(pool.shape[1:]) != (q.shape[2], D, D) or not pool.is_contiguous()
            or pool.dtype not in (torch.float32, torch.bfloat16) or pool.device != q.device):
        raise ValueError(f"pool must be a contiguous float32 or bfloat16 [P, {q.shape[2]}, 128, 128] tensor on q's device")
    if slots is None and pool.shape[0] < d.num_seqs:
        raise ValueError("pool has fewer slots than there are sequences")
    for name, t, n in (("slots", slots, d.num_seqs), ("out_slots", out_slots, q.shape[0] * q.shape[1])):
        if t is not None and (t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or t.device != q.device):
            raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements on q's device")
    if out is not None:
        _check_out("out", out, q.shape, q.device)
    return d


def _recurrent(entry, q, k, v, g, beta, pool, slots, out_slots, cu_seqlens, out, stream):
    d = _check_recurrent(q, k, v, g, beta, pool, slots, out_slots, cu_seqlens, out, entry == "kda_gdn_recurrent")
    with _on(q.device, stream) as s:
        o = out if out is not None else _f32(q)
        _call(entry, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(slots), _ptr(out_slots),
              _ptr(pool), pool.shape[0], KDA_BF16 if pool.dtype == torch.bfloat16 else KDA_F32, _ptr(o),
              ctypes.byref(d), s)
    return o


# ------------------------------------------------------------------ before the rule

def block_in(q: torch.Tensor, k: torch.Tensor, f: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
             dt_bias: _Tensor = None, lower_bound: Optional[float] = None, eps: float = 1e-6,
             stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """The inputs of fwd() from raw projections: q / sqrt(|q|^2 + eps), k alike, the
    gate g from f, and beta = sigmoid(b). With x = f + dt_bias,
    g = -exp(A_log) softplus(x), or with a lower bound (< 0) lower_bound *
    sigmoid(exp(A_log) x). q, k, f [B, T, H, 128] and b [B, T, H] share a dtype (bf16
    or fp32); A_log [H], dt_bias [H, 128] fp32. Returns (q, k, g, beta).
    lower_bound=-5.0 keeps g where fwd() and bwd() are defined. Without a bound nothing
    does: gates of about -5.4 or less over 16 tokens turn fwd()'s results into inf or
    NaN, and -10.9 over eight bwd()'s, without an error (exp(A_log) = 16 and a raw gate
    of 0 give -11). recurrent() takes any gate."""
    return _block_in("kda_block_in", q, k, f, b, A_log, dt_bias, lower_bound, eps, stream)


def gdn_block_in(q: torch.Tensor, k: torch.Tensor, f: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
                 dt_bias: _Tensor = None, lower_bound: Optional[float] = None, eps: float = 1e-6,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """block_in() for gdn_fwd(): f [B, T, H], dt_bias [H], g [B, T, H]. The same holds of
    its gate without a bound."""
    return _block_in("kda_gdn_block_in", q, k, f, b, A_log, dt_bias, lower_bound, eps, stream)


def _rows(name, t, shape, dtype, device, _device=True):
    if (t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device
            or (_device and device.type != "cuda")):
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} device tensor on the first argument's device")


def _rows_desc(x):
    B, T, H, K = x.shape
    return Desc(B, T, H, K, K, B, _DTYPES.get(x.dtype, -1), KDA_F32, None, 0)


def _check_block_in(q, k, f, b, A_log, dt_bias, lower_bound, scalar_gate, _device=True):
    if q.dim() != 4 or q.dtype not in _DTYPES:
        raise ValueError("q must be a bfloat16 or float32 [B, T, H, 128] tensor")
    rows, dtype, device = q.shape, q.dtype, q.device
    heads = rows[:3]
    gate = heads if scalar_gate else rows
    for name, t, shape in (("q", q, rows), ("k", k, rows), ("f", f, gate), ("b", b, heads)):
        _rows(name, t, shape, dtype, device, _device)
    _rows("A_log", A_log, rows[2:3], torch.float32, device, _device)
    if dt_bias is not None:
        _rows("dt_bias", dt_bias, gate[2:], torch.float32, device, _device)
    if lower_bound is not None and not ctypes.c_float(lower_bound).value < 0:
        raise ValueError("lower_bound must be negative (None: no bound)")


def _block_in(entry, q, k, f, b, A_log, dt_bias, lower_bound, eps, stream):
    scalar = entry == "kda_gdn_block_in"
    _check_block_in(q, k, f, b, A_log, dt_bias, lower_bound, scalar)
    with _on(q.device, stream) as s:
        outs = [torch.empty_like(q), torch.empty_like(k), _f32(f), _f32(b)]
        _call(entry, _ptr(q), _ptr(k), _ptr(f), _ptr(b), _ptr(A_log), _ptr(dt_bias), lower_bound or 0.0, eps,
              *map(_ptr, outs), ctypes.byref(_rows_desc(q)), s)
    return tuple(outs)


def block_in_bwd(q: torch.Tensor, k: torch.Tensor, f: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
                 dq: torch.Tensor, dk: torch.Tensor, dg: torch.Tensor, dbeta: torch.Tensor, dt_bias: _Tensor = None,
                 lower_bound: Optional[float] = None, eps: float = 1e-6,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of block_in(): its inputs, and the gradients with respect to its outputs
    (as bwd() returns them). Returns (dq, dk, df, db, dA_log, ddt_bias), the first four
    in q's dtype, the sums over tokens fp32 (ddt_bias None without dt_bias). Every row is
    summed: with packed sequences that end before T, cut all arguments to the first cu[N]
    tokens, since bwd() leaves the rows behind them unset."""
    return _block_in_bwd("kda_block_in_bwd", q, k, f, b, A_log, dq, dk, dg, dbeta, dt_bias, lower_bound, eps, stream)


def gdn_block_in_bwd(q: torch.Tensor, k: torch.Tensor, f: torch.Tensor, b: torch.Tensor, A_log: torch.Tensor,
                     dq: torch.Tensor, dk: torch.Tensor, dg: torch.Tensor, dbeta: torch.Tensor,
                     dt_bias: _Tensor = None, lower_bound: Optional[float] = None, eps: float = 1e-6,
                     stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of gdn_block_in(), as block_in_bwd() (which rows are summed, too)."""
    return _block_in_bwd("kda_gdn_block_in_bwd", q, k, f, b, A_log, dq, dk, dg, dbeta, dt_bias, lower_bound, eps,
                         stream)


def _check_block_in_bwd(q, k, f, b, A_log, dq, dk, dg, dbeta, dt_bias, lower_bound, scalar_gate, _device=True):
    _check_block_in(q, k, f, b, A_log, dt_bias, lower_bound, scalar_gate, _device)
    for name, t, like, dtype in (("dq", dq, q, q.dtype), ("dk", dk, q, q.dtype), ("dg", dg, f, torch.float32),
                                 ("dbeta", dbeta, b, torch.float32)):
        _rows(name, t, like.shape, dtype, q.device, _device)


def _block_in_bwd(entry, q, k, f, b, A_log, dq, dk, dg, dbeta, dt_bias, lower_bound, eps, stream):
    scalar = entry == "kda_gdn_block_in_bwd"
    _check_block_in_bwd(q, k, f, b, A_log, dq, dk, dg, dbeta, dt_bias, lower_bound, scalar)
    d = _rows_desc(q)
    with _on(q.device, stream) as s:
        ws = q.new_empty(int(lib().kda_block_in_bwd_workspace_size(ctypes.byref(d))), dtype=torch.uint8)
        d.workspace, d.workspace_bytes = ws.data_ptr(), ws.numel()
        outs = [torch.empty_like(x) for x in (q, k, f, b, A_log)]
        dbias = torch.empty_like(dt_bias) if dt_bias is not None else None
        _call(entry, _ptr(q), _ptr(k), _ptr(f), _ptr(b), _ptr(A_log), _ptr(dt_bias), lower_bound or 0.0, eps, _ptr(dq),
              _ptr(dk), _ptr(dg), _ptr(dbeta), *map(_ptr, outs), _ptr(dbias), ctypes.byref(d), s)
    return (*outs, dbias)


# ------------------------------------------------------------------- after the rule

def block_out(o: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, activation: str = "sigmoid", eps: float = 1e-5,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Gated RMS norm of fwd()'s output: o / sqrt(mean(o^2) + eps) * weight * act(z), over
    the 128 channels of each (token, head). o fp32, z bf16 or fp32 [B, T, H, 128], weight
    fp32 [128]; activation "sigmoid" or "silu" (z sigmoid(z)). Returns y in z's dtype."""
    _check_block_out(o, z, weight, activation)
    with _on(z.device, stream) as s:
        y = torch.empty_like(z)
        _call("kda_block_out", _ptr(o), _ptr(z), _ptr(weight), eps, ACTIVATIONS[activation], _ptr(y),
              ctypes.byref(_rows_desc(z)), s)
    return y


def _check_block_out(o, z, weight, activation, dy=None, _device=True):
    if z.dim() != 4 or z.dtype not in _DTYPES:
        raise ValueError("z must be a bfloat16 or float32 [B, T, H, 128] tensor")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    _rows("z", z, z.shape, z.dtype, z.device, _device)
    _rows("o", o, z.shape, torch.float32, z.device, _device)
    _rows("weight", weight, (D,), torch.float32, z.device, _device)
    if dy is not None:
        _rows("dy", dy, z.shape, z.dtype, z.device, _device)


def block_out_bwd(o: torch.Tensor, z: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
                  activation: str = "sigmoid", eps: float = 1e-5,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of block_out(). Returns (do fp32, dz in z's dtype, dweight fp32). dweight
    takes every row: cut padded ones off, as for block_in_bwd()."""
    _check_block_out(o, z, weight, activation, dy)
    d = _rows_desc(z)
    with _on(z.device, stream) as s:
        ws = z.new_empty(int(lib().kda_block_out_bwd_workspace_size(ctypes.byref(d))), dtype=torch.uint8)
        d.workspace, d.workspace_bytes = ws.data_ptr(), ws.numel()
        do, dz, dw = torch.empty_like(o), torch.empty_like(z), torch.empty_like(weight)
        _call("kda_block_out_bwd", _ptr(o), _ptr(z), _ptr(weight), eps, ACTIVATIONS[activation], _ptr(dy), _ptr(do),
              _ptr(dz), _ptr(dw), ctypes.byref(d), s)
    return do, dz, dw

"""Torch marshalling of the operators around the rule: its gradient, its recurrent
form over a pool of states, and what comes right before and after it
(include/kda.h). Outputs and workspaces are allocated on the call's stream."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional, Tuple

import torch

from . import D, _check_inputs, _check_out, _check_state, _desc, _ptr
from ._lib import KDAError, lib

_Tensor = Optional[torch.Tensor]


@contextlib.contextmanager
def _on(device: torch.device, stream: Optional[torch.cuda.Stream]):
    """Makes `device` and the call's stream current, so that launches and
    allocations go there; yields the stream as the C ABI takes it."""
    with torch.cuda.device(device):
        s = stream or torch.cuda.current_stream(device)
        if s.device != device:
            raise ValueError("stream must belong to the tensors' device")
        with torch.cuda.stream(s):
            yield ctypes.c_void_p(s.cuda_stream)


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
    d_initial_state): dq, dk, dv in q's dtype, the others fp32. Nothing is kept from
    the forward; states are recomputed. workspace: an optional uint8 device tensor of
    bwd_workspace_size() bytes, used by one call at a time; allocated otherwise."""
    return _bwd("kda_bwd", q, k, v, g, beta, do, cu_seqlens, initial_state, d_final_state, stream, workspace)


def gdn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, do: torch.Tensor,
            cu_seqlens: _Tensor = None, initial_state: _Tensor = None, d_final_state: _Tensor = None,
            stream: Optional[torch.cuda.Stream] = None, workspace: _Tensor = None) -> Tuple[torch.Tensor, ...]:
    """Gradient of gdn_fwd(): as bwd(), with g and dg [B, T, H]."""
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
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        d.workspace = workspace.data_ptr()
        d.workspace_bytes = workspace.numel() * workspace.element_size()
        outs = [torch.empty_like(x) for x in (q, k, v, g, beta)]
        dh0 = torch.empty(sshape, dtype=torch.float32, device=q.device)
        _call(entry, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(initial_state), _ptr(do),
              _ptr(d_final_state), *map(_ptr, outs), _ptr(dh0), ctypes.byref(d), s)
    return (*outs, dh0)

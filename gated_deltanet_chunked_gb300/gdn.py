"""Thin ctypes binding of libgdn.so (include/gdn.h).

Argument marshalling only: every step of the forward runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. There is
no fallback: if libgdn.so cannot be built or loaded, ``load()`` raises.

The entry points keep the C names:
  gdn_chunk_fwd, gdn_chunk_fwd_workspace_size, gdn_recurrent_step,
  gdn_recurrent_step_gated, gdn_gated_rmsnorm, gdn_causal_conv1d_silu,
  gdn_causal_conv1d_silu_step, gdn_gating, gdn_linear_recurrence,
  gdn_linear_recurrence_bwd, gdn_linear_recurrence_step, gdn_layernorm,
  gdn_layernorm_bwd, gdn_gated_rmsnorm_bwd,
  gdn_read_device_status, gdn_get_device_status, gdn_status_string, gdn_version.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import threading
from typing import Optional

import torch

from . import build as _build

GDN_OK, GDN_EINVAL, GDN_EUNSUPPORTED, GDN_ECUDA, GDN_ETIMEOUT, GDN_EDEVICE_INPUT, GDN_ETOOBIG = range(7)
GDN_NOALLOC_SCRATCH_BYTES = 32 << 20
GDN_DT_F32, GDN_DT_BF16 = 0, 1
GDN_FLAG_BETA_BF16, GDN_FLAG_STATE_BF16, GDN_FLAG_GATE_CHANNEL = 1 << 1, 1 << 2, 1 << 3

SYMBOLS = ("gdn_chunk_fwd", "gdn_chunk_fwd_workspace_size", "gdn_recurrent_step", "gdn_read_device_status",
           "gdn_status_string", "gdn_version", "gdn_profile_enable", "gdn_profile_collect", "gdn_kernel_name",
           "gdn_chunk_fwd_noalloc", "gdn_recurrent_step_gated", "gdn_gated_rmsnorm", "gdn_causal_conv1d_silu",
           "gdn_gating", "gdn_causal_conv1d_silu_step", "gdn_chunk_fwd_gated", "gdn_get_device_status",
           "gdn_set_wait_limit_ns", "gdn_linear_recurrence", "gdn_linear_recurrence_states_size",
           "gdn_linear_recurrence_bwd", "gdn_linear_recurrence_step", "gdn_layernorm", "gdn_layernorm_bwd",
           "gdn_layernorm_bwd_workspace_size", "gdn_gated_rmsnorm_bwd", "gdn_gated_rmsnorm_bwd_workspace_size")
GDN_K_COUNT = 18


class GdnProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("seqlen", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("total_tokens", ctypes.c_int32), ("hq", ctypes.c_int32), ("hv", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("num_state_slots", ctypes.c_int32)]


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {gdn_status_string(status)}")


_lib = None
_lock = threading.Lock()
_vp, _fp, _ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p


def load(path: Optional[str] = None):
    """Build (if stale) and load libgdn.so; raises if either step fails."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            lib = ctypes.CDLL(path or _build.build())
            P = ctypes.POINTER(GdnProblem)
            lib.gdn_chunk_fwd.argtypes = [P, _vp, _vp, _vp, _fp, _fp, ctypes.c_float, _fp, _ip, _vp, _fp, _vp,
                                          ctypes.c_size_t, _vp]
            lib.gdn_chunk_fwd.restype = ctypes.c_int
            lib.gdn_chunk_fwd_gated.argtypes = [P, _vp, _vp, _vp, _fp, _fp, ctypes.c_float, _fp, _ip, _vp, _fp,
                                                ctypes.c_float, _vp, _fp, _vp, ctypes.c_size_t, _vp]
            lib.gdn_chunk_fwd_gated.restype = ctypes.c_int
            lib.gdn_chunk_fwd_workspace_size.argtypes = [P]
            lib.gdn_chunk_fwd_workspace_size.restype = ctypes.c_size_t
            lib.gdn_recurrent_step.argtypes = [P, _vp, _vp, _vp, _fp, _fp, ctypes.c_float, _fp, _ip, _vp, _vp]
            lib.gdn_recurrent_step.restype = ctypes.c_int
            lib.gdn_recurrent_step_gated.argtypes = [P, _vp, _vp, _vp, _fp, _fp, _fp, _fp, ctypes.c_float, _fp,
                                                     _ip, _vp, _fp, ctypes.c_float, _vp, _vp]
            lib.gdn_gated_rmsnorm.argtypes = [P, _vp, _vp, _fp, ctypes.c_float, _vp, _vp]
            lib.gdn_gated_rmsnorm.restype = ctypes.c_int
            lib.gdn_causal_conv1d_silu.argtypes = [P, _vp, _fp, _fp, _vp, _ip, _ip, ctypes.c_int, _vp, _vp, _vp, _vp]
            lib.gdn_causal_conv1d_silu.restype = ctypes.c_int
            lib.gdn_causal_conv1d_silu_step.argtypes = [P, _vp, _fp, _fp, _vp, _ip, ctypes.c_int, _vp, _vp, _vp,
                                                        _vp]
            lib.gdn_causal_conv1d_silu_step.restype = ctypes.c_int
            lib.gdn_gating.argtypes = [P, _fp, _fp, _fp, _fp, _fp, _fp, _vp]
            lib.gdn_gating.restype = ctypes.c_int
            lib.gdn_recurrent_step_gated.restype = ctypes.c_int
            lib.gdn_read_device_status.argtypes = [_vp, ctypes.c_int]
            lib.gdn_read_device_status.restype = ctypes.c_int
            lib.gdn_get_device_status.argtypes = [_vp]
            lib.gdn_get_device_status.restype = ctypes.c_int
            lib.gdn_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
            lib.gdn_set_wait_limit_ns.restype = ctypes.c_int
            lib.gdn_status_string.argtypes = [ctypes.c_int]
            lib.gdn_status_string.restype = ctypes.c_char_p
            lib.gdn_version.argtypes = []
            lib.gdn_version.restype = ctypes.c_int
            lib.gdn_profile_enable.argtypes = [ctypes.c_int]
            lib.gdn_profile_enable.restype = ctypes.c_int
            lib.gdn_profile_collect.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int]
            lib.gdn_profile_collect.restype = ctypes.c_int
            lib.gdn_chunk_fwd_noalloc.argtypes = [P, _vp, _vp, _vp, _fp, _fp, ctypes.c_float, _fp, _ip, _vp, _fp,
                                                  _vp]
            lib.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
            cf, sz = ctypes.c_float, ctypes.c_size_t
            for name, res, args in (
                    ("gdn_linear_recurrence", ctypes.c_int, [P, _vp, _vp, _fp, _ip, _vp, _fp, _fp, _vp]),
                    ("gdn_linear_recurrence_states_size", sz, [P]),
                    ("gdn_linear_recurrence_bwd", ctypes.c_int,
                     [P, _vp, _vp, _vp, _fp, _fp, _fp, _ip, _vp, _vp, _fp, _vp]),
                    ("gdn_linear_recurrence_step", ctypes.c_int, [P, _vp, _vp, _fp, _ip, _vp, _vp]),
                    ("gdn_layernorm", ctypes.c_int, [P, _vp, _fp, _fp, cf, _vp, _fp, _fp, _vp]),
                    ("gdn_layernorm_bwd", ctypes.c_int,
                     [P, _vp, _vp, _fp, _fp, _fp, _vp, _fp, _fp, _vp, sz, _vp]),
                    ("gdn_layernorm_bwd_workspace_size", sz, [P]),
                    ("gdn_gated_rmsnorm_bwd", ctypes.c_int,
                     [P, _vp, _vp, _vp, _fp, cf, _vp, _vp, _fp, _vp, sz, _vp]),
                    ("gdn_gated_rmsnorm_bwd_workspace_size", sz, [P])):
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            lib.gdn_kernel_name.argtypes = [ctypes.c_int]
            lib.gdn_kernel_name.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def lib():
    return load()


def gdn_status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def gdn_version() -> int:
    return int(load().gdn_version())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libgdn wants contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _io_type(dtype) -> int:
    if dtype == torch.float32:
        return GDN_DT_F32
    if dtype == torch.bfloat16:
        return GDN_DT_BF16
    raise ValueError(f"unsupported io dtype {dtype}")


def _io_dtype(t: torch.Tensor) -> int:
    return _io_type(t.dtype)


def _want(dtype, **tensors):
    """Raises ValueError unless every given (non-None) tensor has ``dtype``."""
    for name, t in tensors.items():
        if t is not None and t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _stream(stream, device=None) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


@contextlib.contextmanager
def _launching(stream, dev):
    """Makes ``dev`` and, if given, ``stream`` current: what a call allocates
    then belongs to the stream it runs on, so that PyTorch's allocator hands
    none of it to other work too early."""
    if dev.type != "cuda":
        raise ValueError(f"libgdn wants CUDA tensors, got a tensor on {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            handle = _stream(stream).value or 0
            stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, expected {dev} (the device of the first input)")
        with torch.cuda.stream(stream):
            yield


def _on_device(dev: torch.device, **tensors):
    """Raises ValueError unless every given (non-None) tensor is a CUDA tensor
    on ``dev``. The library reads its device status word and its no-alloc
    scratch on the current device, and the kernels dereference the pointers
    they are given, so a host tensor or a tensor on another GPU must never
    reach it."""
    if dev.type != "cuda":
        raise ValueError(f"libgdn wants CUDA tensors, got a tensor on {dev}")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev} (the device of the first input)")


def _shape(name, t, *shape):
    """Raises ValueError unless tensor ``t`` (if given) has exactly ``shape``."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def prefill_problem(q: torch.Tensor, v: torch.Tensor, num_seqs: int, packed: bool) -> GdnProblem:
    """Descriptor for q [T_total, Hq, dk] (packed) or [B, T, Hq, dk] (dense)."""
    if packed:
        Ttot, hq, dk = q.shape
        batch, seqlen = 1, 0
    else:
        batch, seqlen, hq, dk = q.shape
        Ttot = batch * seqlen
        num_seqs = batch
    return GdnProblem(batch, seqlen, num_seqs, Ttot, hq, v.shape[-2], dk, v.shape[-1], _io_dtype(q), 0, 0)


def gdn_chunk_fwd_workspace_size(problem: GdnProblem) -> int:
    return int(load().gdn_chunk_fwd_workspace_size(ctypes.byref(problem)))


def _prefill_checks(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, z=None, norm_weight=None,
                    workspace=None):
    """Device, dtype and shape checks shared by the prefill wrappers; returns
    (problem, device)."""
    packed = cu_seqlens is not None
    if q.dim() != (3 if packed else 4):
        raise ValueError("q must be [T, Hq, dk] with cu_seqlens, else [B, T, Hq, dk]")
    num_seqs = cu_seqlens.numel() - 1 if packed else q.shape[0]
    dev = q.device
    _want(q.dtype, k=k, v=v, out=out, z=z)
    _want(torch.float32, g=g, beta=beta, initial_state=initial_state, final_state=final_state,
          norm_weight=norm_weight)
    _want(torch.int32, cu_seqlens=cu_seqlens)
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    prob = prefill_problem(q, v, num_seqs, packed)
    lead = q.shape[:-2]  # (T,) packed or (B, T) dense
    _shape("k", k, *q.shape)
    _shape("v", v, *lead, prob.hv, prob.dv)
    _shape("g", g, *lead, prob.hv)
    _shape("beta", beta, *lead, prob.hv)
    _shape("out", out, *v.shape)
    _shape("z", z, *v.shape)
    _shape("norm_weight", norm_weight, prob.dv)
    _shape("initial_state", initial_state, prob.num_seqs, prob.hv, prob.dk, prob.dv)
    _shape("final_state", final_state, prob.num_seqs, prob.hv, prob.dk, prob.dv)
    if packed and cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor [N + 1]")
    _on_device(dev, k=k, v=v, g=g, beta=beta, initial_state=initial_state, cu_seqlens=cu_seqlens, out=out,
               final_state=final_state, z=z, norm_weight=norm_weight, workspace=workspace)
    return prob, dev


def gdn_chunk_fwd(q, k, v, g, beta, scale, initial_state=None, cu_seqlens=None, out=None,
                  final_state=None, output_final_state=True, workspace=None, stream=None,
                  z=None, norm_weight=None, norm_eps=1e-6):
    """Chunked prefill. Packed when ``cu_seqlens`` (int32 device [N+1]) is given.

    Returns (out, final_state). ``workspace`` (uint8 device tensor) is
    allocated with PyTorch when not supplied. With ``z`` (like v) and
    ``norm_weight`` [128] f32, out holds the output gate applied to the
    read-out (gdn_chunk_fwd_gated). Every tensor must sit on q's device; the
    call runs with that device current, on its current stream unless
    ``stream`` is given.
    """
    prob, dev = _prefill_checks(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state, z, norm_weight,
                                workspace)
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=dev)
        if final_state is None and output_final_state:
            final_state = torch.empty((prob.num_seqs, prob.hv, prob.dk, prob.dv), dtype=torch.float32, device=dev)
        need = gdn_chunk_fwd_workspace_size(prob)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        if z is None:
            st = load().gdn_chunk_fwd(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      ctypes.c_float(scale), _ptr(initial_state), _ptr(cu_seqlens), _ptr(out),
                                      _ptr(final_state), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                                      _stream(stream, dev))
            where = "gdn_chunk_fwd"
        else:
            if norm_weight is None:
                raise ValueError("the output gate needs norm_weight")
            st = load().gdn_chunk_fwd_gated(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                            ctypes.c_float(scale), _ptr(initial_state), _ptr(cu_seqlens), _ptr(z),
                                            _ptr(norm_weight), ctypes.c_float(norm_eps), _ptr(out),
                                            _ptr(final_state), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                                            _stream(stream, dev))
            where = "gdn_chunk_fwd_gated"
    if st != GDN_OK:
        raise GdnError(st, where)
    return out, final_state


def gdn_chunk_fwd_noalloc(q, k, v, g, beta, scale, out, final_state=None, initial_state=None, cu_seqlens=None,
                          stream=None):
    """gdn_chunk_fwd without a workspace, for callers that cannot allocate:
    the library uses its fixed device scratch array (GDN_NOALLOC_SCRATCH_BYTES)
    and allocates nothing. ``out`` (and ``final_state`` if wanted) must be
    supplied. Raises GdnError(GDN_ETOOBIG) for problems above that size."""
    if out is None:
        raise ValueError("gdn_chunk_fwd_noalloc writes into a caller-supplied out")
    prob, dev = _prefill_checks(q, k, v, g, beta, initial_state, cu_seqlens, out, final_state)
    with torch.cuda.device(dev):
        st = load().gdn_chunk_fwd_noalloc(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                          ctypes.c_float(scale), _ptr(initial_state), _ptr(cu_seqlens), _ptr(out),
                                          _ptr(final_state), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_chunk_fwd_noalloc")
    return out, final_state


def _decode_flags(state, beta_bf16):
    return (GDN_FLAG_STATE_BF16 if state.dtype == torch.bfloat16 else 0) | (GDN_FLAG_BETA_BF16 if beta_bf16 else 0)


def _decode_checks(q, v, state, state_indices, out, z=None):
    """Shape checks shared by the decode wrappers: q, k [N, Hq, 128],
    v, out, z [N, Hv, 128], state [slots, Hv, 128, 128], state_indices [N]."""
    if q.dim() != 3 or v.dim() != 3 or v.shape[0] != q.shape[0]:
        raise ValueError("q must be [N, Hq, dk] and v [N, Hv, dv] with the same N")
    if state.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"state must be float32 or bfloat16, got {state.dtype}")
    N, hv, dv = v.shape
    if state.dim() != 4 or tuple(state.shape[1:]) != (hv, q.shape[2], dv):
        raise ValueError(f"state must be [slots, {hv}, {q.shape[2]}, {dv}], got {tuple(state.shape)}")
    _shape("out", out, *v.shape)
    _shape("z", z, *v.shape)
    _shape("state_indices", state_indices, N)


def gdn_recurrent_step(q, k, v, g, beta, scale, state, state_indices=None, out=None, stream=None,
                       beta_bf16=False):
    """One decode step; ``state`` [slots, Hv, 128, 128] (f32, or bf16 for a
    bf16 state cache) is updated in place. ``beta_bf16`` rounds beta to bf16."""
    dev = q.device
    _want(q.dtype, k=k, v=v, out=out)
    _want(torch.float32, g=g, beta=beta)
    _want(torch.int32, state_indices=state_indices)
    _decode_checks(q, v, state, state_indices, out)
    N, hq, dk = q.shape
    _shape("k", k, *q.shape)
    _shape("g", g, N, v.shape[1])
    _shape("beta", beta, N, v.shape[1])
    _on_device(dev, k=k, v=v, g=g, beta=beta, state=state, state_indices=state_indices, out=out)
    prob = GdnProblem(N, 1, N, N, hq, v.shape[1], dk, v.shape[2], _io_dtype(q), _decode_flags(state, beta_bf16),
                      state.shape[0])
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=dev)
        st = load().gdn_recurrent_step(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                       ctypes.c_float(scale), _ptr(state), _ptr(state_indices), _ptr(out),
                                       _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_recurrent_step")
    return out


def gdn_recurrent_step_gated(q, k, v, a, b, A_log, dt_bias, scale, state, state_indices=None, out=None,
                             stream=None, z=None, norm_weight=None, norm_eps=1e-6, beta_bf16=False):
    """Decode step from raw q/k and the gate projections a, b [N, Hv] with
    per-head A_log, dt_bias [Hv] (all f32); ``state`` is updated in place.
    With ``z`` [N, Hv, 128] and ``norm_weight`` [128] f32 the output gate
    (head-wise RMSNorm, then silu(z)) is applied before the store. A bf16
    ``state`` is a bf16 state cache; ``beta_bf16`` rounds beta to bf16."""
    dev = q.device
    _want(q.dtype, k=k, v=v, out=out, z=z)
    _want(torch.float32, a=a, b=b, A_log=A_log, dt_bias=dt_bias, norm_weight=norm_weight)
    _want(torch.int32, state_indices=state_indices)
    _decode_checks(q, v, state, state_indices, out, z)
    N, hq, dk = q.shape
    hv = v.shape[1]
    _shape("k", k, *q.shape)
    _shape("a", a, N, hv)
    _shape("b", b, N, hv)
    _shape("A_log", A_log, hv)
    _shape("dt_bias", dt_bias, hv)
    _shape("norm_weight", norm_weight, v.shape[2])
    if z is not None and norm_weight is None:
        raise ValueError("the output gate needs norm_weight")
    _on_device(dev, k=k, v=v, a=a, b=b, A_log=A_log, dt_bias=dt_bias, state=state, state_indices=state_indices,
               out=out, z=z, norm_weight=norm_weight)
    prob = GdnProblem(N, 1, N, N, hq, hv, dk, v.shape[2], _io_dtype(q), _decode_flags(state, beta_bf16),
                      state.shape[0])
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(v.shape, dtype=v.dtype, device=dev)
        st = load().gdn_recurrent_step_gated(ctypes.byref(prob), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b),
                                             _ptr(A_log), _ptr(dt_bias), ctypes.c_float(scale), _ptr(state),
                                             _ptr(state_indices), _ptr(z), _ptr(norm_weight),
                                             ctypes.c_float(norm_eps), _ptr(out), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_recurrent_step_gated")
    return out


def gdn_gated_rmsnorm(o, z, weight, eps, out=None, stream=None):
    """y = o / sqrt(mean(o^2) + eps) * weight * silu(z) per (token, head) row
    of o, z [T, Hv, 128] (io dtype) with weight [128] f32. ``out`` may be o."""
    dev = o.device
    if o.dim() != 3:
        raise ValueError("o must be [T, Hv, 128]")
    T, hv, dv = o.shape
    _want(o.dtype, z=z, out=out)
    _want(torch.float32, weight=weight)
    _shape("z", z, *o.shape)
    _shape("out", out, *o.shape)
    _shape("weight", weight, dv)
    _on_device(dev, z=z, weight=weight, out=out)
    prob = GdnProblem(1, 0, 1, T, 1, hv, dv, dv, _io_dtype(o), 0, 0)
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty_like(o)
        st = load().gdn_gated_rmsnorm(ctypes.byref(prob), _ptr(o), _ptr(z), _ptr(weight), ctypes.c_float(eps),
                                      _ptr(out), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_gated_rmsnorm")
    return out


def _conv_checks(x, weight, bias, conv_state, state_indices, cu_seqlens, q, k, v, hq, hv, N):
    dev = x.device
    if x.dim() != 2:
        raise ValueError("x must be [T, C]")
    T, C = x.shape
    if C != (2 * hq + hv) * 128:
        raise ValueError("x must have (2 hq + hv) * 128 channels")
    _want(x.dtype, conv_state=conv_state, q=q, k=k, v=v)
    _want(torch.float32, weight=weight, bias=bias)
    _want(torch.int32, state_indices=state_indices, cu_seqlens=cu_seqlens)
    _shape("weight", weight, C, 4)
    _shape("bias", bias, C)
    _shape("state_indices", state_indices, N)
    _shape("cu_seqlens", cu_seqlens, N + 1)
    _shape("q", q, T, hq, 128)
    _shape("k", k, T, hq, 128)
    _shape("v", v, T, hv, 128)
    if conv_state is not None and (conv_state.dim() != 3 or tuple(conv_state.shape[1:]) != (3, C)):
        raise ValueError(f"conv_state must be [slots, 3, {C}], got {tuple(conv_state.shape)}")
    _on_device(dev, weight=weight, bias=bias, conv_state=conv_state, state_indices=state_indices,
               cu_seqlens=cu_seqlens, q=q, k=k, v=v)
    return dev


def gdn_causal_conv1d_silu(x, weight, hq, hv, bias=None, conv_state=None, state_indices=None, cu_seqlens=None,
                           norm_qk=False, q=None, k=None, v=None, stream=None):
    """Short causal convolution (4 taps, weight [C, 4] f32 oldest first) + SiLU
    over packed tokens x [T, C] (C = (2 hq + hv) * 128), split into q, k
    [T, hq, 128] and v [T, hv, 128]; ``conv_state`` [slots, 3, C] is read and
    updated in place. ``norm_qk`` L2-normalises every q and k head row."""
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    dev = _conv_checks(x, weight, bias, conv_state, state_indices, cu_seqlens, q, k, v, hq, hv, N)
    T = x.shape[0]
    slots = 0 if conv_state is None else conv_state.shape[0]
    prob = GdnProblem(1, 0, N, T, hq, hv, 128, 128, _io_dtype(x), 0, slots)
    with torch.cuda.device(dev):
        q = torch.empty((T, hq, 128), dtype=x.dtype, device=dev) if q is None else q
        k = torch.empty((T, hq, 128), dtype=x.dtype, device=dev) if k is None else k
        v = torch.empty((T, hv, 128), dtype=x.dtype, device=dev) if v is None else v
        st = load().gdn_causal_conv1d_silu(ctypes.byref(prob), _ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state),
                                           _ptr(state_indices), _ptr(cu_seqlens), int(bool(norm_qk)), _ptr(q),
                                           _ptr(k), _ptr(v), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_causal_conv1d_silu")
    return q, k, v


def gdn_causal_conv1d_silu_step(x, weight, hq, hv, bias=None, conv_state=None, state_indices=None, norm_qk=False,
                                q=None, k=None, v=None, stream=None):
    """gdn_causal_conv1d_silu for one token per sequence: x [N, C]."""
    N = x.shape[0]
    dev = _conv_checks(x, weight, bias, conv_state, state_indices, None, q, k, v, hq, hv, N)
    slots = 0 if conv_state is None else conv_state.shape[0]
    prob = GdnProblem(N, 1, N, N, hq, hv, 128, 128, _io_dtype(x), 0, slots)
    with torch.cuda.device(dev):
        q = torch.empty((N, hq, 128), dtype=x.dtype, device=dev) if q is None else q
        k = torch.empty((N, hq, 128), dtype=x.dtype, device=dev) if k is None else k
        v = torch.empty((N, hv, 128), dtype=x.dtype, device=dev) if v is None else v
        st = load().gdn_causal_conv1d_silu_step(ctypes.byref(prob), _ptr(x), _ptr(weight), _ptr(bias),
                                                _ptr(conv_state), _ptr(state_indices), int(bool(norm_qk)), _ptr(q),
                                                _ptr(k), _ptr(v), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_causal_conv1d_silu_step")
    return q, k, v


def gdn_gating(a, b, A_log, dt_bias, g=None, beta=None, stream=None):
    """g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b), a, b [T, Hv] f32."""
    dev = a.device
    if a.dim() != 2:
        raise ValueError("a must be [T, Hv]")
    T, hv = a.shape
    _want(torch.float32, a=a, b=b, A_log=A_log, dt_bias=dt_bias, g=g, beta=beta)
    for name, t in (("b", b), ("g", g), ("beta", beta)):
        _shape(name, t, T, hv)
    _shape("A_log", A_log, hv)
    _shape("dt_bias", dt_bias, hv)
    _on_device(dev, b=b, A_log=A_log, dt_bias=dt_bias, g=g, beta=beta)
    prob = GdnProblem(1, 0, 1, T, 1, hv, 128, 128, GDN_DT_F32, 0, 0)
    with torch.cuda.device(dev):
        g = torch.empty_like(a) if g is None else g
        beta = torch.empty_like(a) if beta is None else beta
        st = load().gdn_gating(ctypes.byref(prob), _ptr(a), _ptr(b), _ptr(A_log), _ptr(dt_bias), _ptr(g),
                               _ptr(beta), _stream(stream, dev))
    if st != GDN_OK:
        raise GdnError(st, "gdn_gating")
    return g, beta


def _arg(name, t, dtype, shape, dev):
    """Address of tensor ``t`` (None: None) after the checks of its type,
    shape, device and layout: ValueError before any call."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev} (the device of the first input)")
    raise ValueError(f"{name} must be contiguous")


def _first(name, t):
    """Address of the tensor that the others are checked against."""
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _descriptor(*fields):
    """A problem descriptor and the reference that calls take (never written to)."""
    prob = GdnProblem(*fields)
    return prob, ctypes.byref(prob)


def _elsewhere(dev, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    return stream is not None or (dev.type == "cuda" and dev.index != torch.cuda.current_device())


def _current(dev) -> int:
    """Handle of the current stream of ``dev``, the current device."""
    if dev.type != "cuda":
        raise ValueError(f"libgdn wants CUDA tensors, got a tensor on {dev}")
    return torch._C._cuda_getCurrentRawStream(dev.index)


@functools.lru_cache(maxsize=1024)
def _linrec_layout(shape, dtype, gate_dims, offsets):
    """(descriptor's reference, state shape, states shape, gate's type and
    shape) of the recurrence on x of ``shape``, [T, Hv, 128] with cu_seqlens of
    shape ``offsets`` or [B, T, Hv, 128] with None."""
    packed = offsets is not None
    if len(shape) != (3 if packed else 4):
        raise ValueError("x must be [T, Hv, 128] with cu_seqlens, else [B, T, Hv, 128]")
    if packed and len(offsets) != 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor [N + 1]")
    if packed:
        total, hv, dv = shape
        batch, seqlen, num_seqs = 1, 0, offsets[0] - 1
    else:
        batch, seqlen, hv, dv = shape
        total, num_seqs = batch * seqlen, batch
    channel = gate_dims == len(shape)
    _, ref = _descriptor(batch, seqlen, num_seqs, total, hv, hv, dv, dv, _io_type(dtype),
                         GDN_FLAG_GATE_CHANNEL if channel else 0, 0)
    gate = (dtype, shape) if channel else (torch.float32, shape[:-1])
    return ref, (num_seqs, hv, dv), ((total + 63) // 64, hv, dv), gate


def gdn_linear_recurrence(x, g, initial_state=None, cu_seqlens=None, out=None, final_state=None,
                          output_final_state=True, save_states=False, states=None, stream=None):
    """s_t = exp(g_t) s_{t-1} + x_t per channel, out = s: x [T, Hv, 128] packed
    by ``cu_seqlens`` (int32 [N + 1]) or [B, T, Hv, 128]; the log-decays g <= 0
    per head ([T, Hv] f32, as gdn_gating gives them) or per channel (x's shape
    and type). ``initial_state`` and the returned final state are
    [N, Hv, 128] f32.

    Returns (out, final_state), and with ``save_states`` (or ``states`` given)
    also the states that gdn_linear_recurrence_bwd starts from,
    [ceil(T / 64), Hv, 128] f32 over all T rows."""
    dev = x.device
    if _elsewhere(dev, stream):
        with _launching(stream, dev):
            return gdn_linear_recurrence(x, g, initial_state, cu_seqlens, out, final_state, output_final_state,
                                         save_states, states)
    ref, state_shape, states_shape, gate = _linrec_layout(
        x.shape, x.dtype, g.dim(), None if cu_seqlens is None else cu_seqlens.shape)
    f32 = torch.float32
    px = _first("x", x)
    pg = _arg("g", g, *gate, dev)
    ps0 = _arg("initial_state", initial_state, f32, state_shape, dev)
    pcu = _arg("cu_seqlens", cu_seqlens, torch.int32, (state_shape[0] + 1,), dev)
    po = _arg("out", out, x.dtype, x.shape, dev)
    pf = _arg("final_state", final_state, f32, state_shape, dev)
    pst = _arg("states", states, f32, states_shape, dev)
    handle = _current(dev)
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    if final_state is None and output_final_state:
        final_state = torch.empty(state_shape, dtype=f32, device=dev)
        pf = final_state.data_ptr()
    if states is None and save_states:
        states = torch.empty(states_shape, dtype=f32, device=dev)
        pst = states.data_ptr()
    st = load().gdn_linear_recurrence(ref, px, pg, ps0, pcu, po, pf, pst, handle)
    if st != GDN_OK:
        raise GdnError(st, "gdn_linear_recurrence")
    return (out, final_state) if states is None else (out, final_state, states)


def gdn_linear_recurrence_bwd(dout, x, g, states, initial_state=None, cu_seqlens=None, dfinal_state=None, dx=None,
                              dg=None, dinitial_state=None, stream=None):
    """Backward pass of gdn_linear_recurrence from the gradients of out and of
    the final state (None: zeros), with ``states`` of the forward pass.
    Returns (dx, dg, dinitial_state); dinitial_state is None unless an
    ``initial_state`` or a dinitial_state to write is given."""
    dev = x.device
    if _elsewhere(dev, stream):
        with _launching(stream, dev):
            return gdn_linear_recurrence_bwd(dout, x, g, states, initial_state, cu_seqlens, dfinal_state, dx, dg,
                                             dinitial_state)
    if states is None:
        raise ValueError("the backward pass needs the forward pass's states (save_states=True)")
    ref, state_shape, states_shape, gate = _linrec_layout(
        x.shape, x.dtype, g.dim(), None if cu_seqlens is None else cu_seqlens.shape)
    f32 = torch.float32
    px = _first("x", x)
    pdo = _arg("dout", dout, x.dtype, x.shape, dev)
    pg = _arg("g", g, *gate, dev)
    pst = _arg("states", states, f32, states_shape, dev)
    ps0 = _arg("initial_state", initial_state, f32, state_shape, dev)
    pcu = _arg("cu_seqlens", cu_seqlens, torch.int32, (state_shape[0] + 1,), dev)
    pdf = _arg("dfinal_state", dfinal_state, f32, state_shape, dev)
    pdx = _arg("dx", dx, x.dtype, x.shape, dev)
    pdg = _arg("dg", dg, *gate, dev)
    pd0 = _arg("dinitial_state", dinitial_state, f32, state_shape, dev)
    handle = _current(dev)
    if dx is None:
        dx = torch.empty_like(x)
        pdx = dx.data_ptr()
    if dg is None:
        dg = torch.empty_like(g)
        pdg = dg.data_ptr()
    if dinitial_state is None and initial_state is not None:
        dinitial_state = torch.empty(state_shape, dtype=f32, device=dev)
        pd0 = dinitial_state.data_ptr()
    st = load().gdn_linear_recurrence_bwd(ref, pdo, px, pg, pst, ps0, pdf, pcu, pdx, pdg, pd0, handle)
    if st != GDN_OK:
        raise GdnError(st, "gdn_linear_recurrence_bwd")
    return dx, dg, dinitial_state


def gdn_linear_recurrence_step(x, g, state, state_indices=None, out=None, stream=None):
    """One decode token per sequence: x [N, Hv, 128]; ``state``
    [slots, Hv, 128] f32 is updated in place at ``state_indices`` (int32 [N];
    None: slot n; negative: skipped, its out rows are not written)."""
    dev = x.device
    if _elsewhere(dev, stream):
        with _launching(stream, dev):
            return gdn_linear_recurrence_step(x, g, state, state_indices, out)
    if x.dim() != 3 or state.dim() != 3:
        raise ValueError("x must be [N, Hv, 128] and state [slots, Hv, 128]")
    N, hv, dv = x.shape
    slots = state.shape[0]
    channel = g.dim() == 3
    px = _first("x", x)
    pg = _arg("g", g, x.dtype if channel else torch.float32, x.shape if channel else (N, hv), dev)
    ps = _arg("state", state, torch.float32, (slots, hv, dv), dev)
    pi = _arg("state_indices", state_indices, torch.int32, (N,), dev)
    po = _arg("out", out, x.dtype, x.shape, dev)
    _, ref = _descriptor(N, 1, N, N, hv, hv, dv, dv, _io_dtype(x), GDN_FLAG_GATE_CHANNEL if channel else 0, slots)
    handle = _current(dev)
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    st = load().gdn_linear_recurrence_step(ref, px, pg, ps, pi, po, handle)
    if st != GDN_OK:
        raise GdnError(st, "gdn_linear_recurrence_step")
    return out


@functools.lru_cache(maxsize=1024)
def _rows_descriptor(shape, dtype):
    """(descriptor's reference, leading shape, width) of a row-wise norm over the last dimension."""
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError("the last dimension must not be empty")
    width, rows = shape[-1], shape[:-1].numel()
    if rows >= 1 << 31:
        raise ValueError("too many rows")
    return _descriptor(1, 0, 1, rows, 1, 1, width, width, _io_type(dtype), 0, 0)[1], shape[:-1], width


def gdn_layernorm(x, weight=None, bias=None, eps=1e-5, out=None, save_stats=False, mean=None, rstd=None,
                  stream=None):
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last dimension
    of x (1 to 16384 wide); weight and bias [D] f32 or None. ``out`` may be x.
    Returns y, and with ``save_stats`` (y, mean, rstd), the last two f32 of
    x's leading shape, for gdn_layernorm_bwd."""
    dev = x.device
    if _elsewhere(dev, stream):
        with _launching(stream, dev):
            return gdn_layernorm(x, weight, bias, eps, out, save_stats, mean, rstd)
    ref, lead, width = _rows_descriptor(x.shape, x.dtype)
    f32 = torch.float32
    px = _first("x", x)
    pw = _arg("weight", weight, f32, (width,), dev)
    pb = _arg("bias", bias, f32, (width,), dev)
    po = _arg("out", out, x.dtype, x.shape, dev)
    pm = _arg("mean", mean, f32, lead, dev)
    pr = _arg("rstd", rstd, f32, lead, dev)
    handle = _current(dev)
    if out is None:
        out = torch.empty_like(x)
        po = out.data_ptr()
    if save_stats:
        if mean is None:
            mean = torch.empty(lead, dtype=f32, device=dev)
            pm = mean.data_ptr()
        if rstd is None:
            rstd = torch.empty_like(mean)
            pr = rstd.data_ptr()
    st = load().gdn_layernorm(ref, px, pw, pb, eps, po, pm, pr, handle)
    if st != GDN_OK:
        raise GdnError(st, "gdn_layernorm")
    return (out, mean, rstd) if save_stats else out


def _workspace(workspace, need, dev):
    """(address, bytes, tensor) of the caller's uint8 workspace, or of one of
    ``need`` bytes."""
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        return workspace.data_ptr(), max(need, 256), workspace
    if workspace.dtype != torch.uint8:
        raise ValueError("workspace must be a uint8 tensor")
    return _arg("workspace", workspace, torch.uint8, workspace.shape, dev), workspace.numel(), workspace


def gdn_layernorm_bwd(dy, x, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, need_dweight=True,
                      need_dbias=True, workspace=None, stream=None):
    """Backward pass of gdn_layernorm with the forward pass's mean and rstd.
    Returns (dx, dweight, dbias), the last two [D] f32 sums over all rows (None
    where not needed). ``dx`` may be dy or x. ``workspace`` (uint8, of
    gdn_layernorm_bwd_workspace_size bytes) is allocated when not supplied."""
    dev = x.device
    if _elsewhere(dev, stream):
        with _launching(stream, dev):
            return gdn_layernorm_bwd(dy, x, mean, rstd, weight, dx, dweight, dbias, need_dweight, need_dbias,
                                     workspace)
    ref, lead, width = _rows_descriptor(x.shape, x.dtype)
    f32 = torch.float32
    px = _first("x", x)
    pdy = _arg("dy", dy, x.dtype, x.shape, dev)
    pm = _arg("mean", mean, f32, lead, dev)
    pr = _arg("rstd", rstd, f32, lead, dev)
    pw = _arg("weight", weight, f32, (width,), dev)
    pdx = _arg("dx", dx, x.dtype, x.shape, dev)
    pdw = _arg("dweight", dweight, f32, (width,), dev)
    pdb = _arg("dbias", dbias, f32, (width,), dev)
    handle = _current(dev)
    if dx is None:
        dx = torch.empty_like(x)
        pdx = dx.data_ptr()
    if dweight is None and need_dweight:
        dweight = torch.empty(width, dtype=f32, device=dev)
        pdw = dweight.data_ptr()
    if dbias is None and need_dbias:
        dbias = torch.empty(width, dtype=f32, device=dev)
        pdb = dbias.data_ptr()
    lib, pws, nbytes = load(), None, 0
    if pdw or pdb or workspace is not None:
        pws, nbytes, workspace = _workspace(workspace, lib.gdn_layernorm_bwd_workspace_size(ref), dev)
    st = lib.gdn_layernorm_bwd(ref, pdy, px, pm, pr, pw, pdx, pdw, pdb, pws, nbytes, handle)
    if st != GDN_OK:
        raise GdnError(st, "gdn_layernorm_bwd")
    return dx, dweight, dbias


def gdn_gated_rmsnorm_bwd(dy, o, z, weight, eps, do=None, dz=None, dweight=None, need_dweight=True, workspace=None,
                          stream=None):
    """Backward pass of gdn_gated_rmsnorm: dy, o, z [T, Hv, 128], weight [128]
    f32. Returns (do, dz, dweight); dweight [128] f32 sums over all (token,
    head) rows (None where not needed). do and dz may be any of dy, o and z.
    ``workspace`` (uint8, of gdn_gated_rmsnorm_bwd_workspace_size bytes) is
    allocated when not supplied."""
    dev = o.device
    if _elsewhere(dev, stream):
        with _launching(stream, dev):
            return gdn_gated_rmsnorm_bwd(dy, o, z, weight, eps, do, dz, dweight, need_dweight, workspace)
    if o.dim() != 3:
        raise ValueError("o must be [T, Hv, 128]")
    T, hv, dv = shape = o.shape
    f32, io = torch.float32, o.dtype
    po = _first("o", o)
    pdy = _arg("dy", dy, io, shape, dev)
    pz = _arg("z", z, io, shape, dev)
    pw = _arg("weight", weight, f32, (dv,), dev)
    pdo = _arg("do", do, io, shape, dev)
    pdz = _arg("dz", dz, io, shape, dev)
    pdw = _arg("dweight", dweight, f32, (dv,), dev)
    _, ref = _descriptor(1, 0, 1, T, 1, hv, dv, dv, _io_dtype(o), 0, 0)
    handle = _current(dev)
    if do is None:
        do = torch.empty_like(o)
        pdo = do.data_ptr()
    if dz is None:
        dz = torch.empty_like(o)
        pdz = dz.data_ptr()
    if dweight is None and need_dweight:
        dweight = torch.empty(dv, dtype=f32, device=dev)
        pdw = dweight.data_ptr()
    lib, pws, nbytes = load(), None, 0
    if pdw or workspace is not None:
        pws, nbytes, workspace = _workspace(workspace, lib.gdn_gated_rmsnorm_bwd_workspace_size(ref), dev)
    st = lib.gdn_gated_rmsnorm_bwd(ref, pdy, po, pz, pw, eps, pdo, pdz, pdw, pws, nbytes, handle)
    if st != GDN_OK:
        raise GdnError(st, "gdn_gated_rmsnorm_bwd")
    return do, dz, dweight


def gdn_read_device_status(stream=None, clear: bool = True) -> int:
    """Synchronises ``stream`` (the current device's current stream when
    None) and returns the device status word, clearing it when ``clear``."""
    return int(load().gdn_read_device_status(_stream(stream), int(clear)))


def gdn_get_device_status(stream=None) -> int:
    """gdn_read_device_status with clear: returns the first device-side error
    recorded since the last read and resets the word (cudaGetLastError-like)."""
    return int(load().gdn_get_device_status(_stream(stream)))


def gdn_set_wait_limit_ns(ns: int) -> None:
    """Limit of the kernels' bounded device-side waits for later launches
    (0 restores the default 2 s); for tests of the timeout path."""
    load().gdn_set_wait_limit_ns(int(ns))


def gdn_profile_enable(enable: bool = True) -> None:
    load().gdn_profile_enable(int(enable))


def gdn_kernel_name(kernel: int) -> str:
    return load().gdn_kernel_name(int(kernel)).decode()


def gdn_profile_collect(reset: bool = True) -> dict:
    """{kernel name: (launches, summed event ms, timed launches)} for kernels that ran."""
    n = GDN_K_COUNT
    launches = (ctypes.c_longlong * n)()
    ms = (ctypes.c_double * n)()
    timed = (ctypes.c_longlong * n)()
    st = load().gdn_profile_collect(ctypes.cast(launches, _vp), ctypes.cast(ms, _vp), ctypes.cast(timed, _vp), n,
                                    int(reset))
    if st != GDN_OK:
        raise GdnError(st, "gdn_profile_collect")
    return {gdn_kernel_name(i): (int(launches[i]), float(ms[i]), int(timed[i])) for i in range(n) if launches[i]}

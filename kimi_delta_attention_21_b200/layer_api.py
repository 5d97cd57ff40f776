"""Torch-facing binding of the operators around the gated delta rule: argument marshalling only.

The norm of queries and keys with the rotation by position and its gradients;
the gated delta rule token by token and its gradients; the output path in e4m3.
Every step runs inside libkda's CUDA kernels, on the current stream of the
tensors' device (which need not be the current device).
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import GdnDecodeArgs, QkNormArgs, QkNormBwdArgs, RecBwdArgs, check
from .api import _DT

NORMS = {"l2": _lib.NORM_L2, "rms": _lib.NORM_RMS}


# These calls can take a few microseconds on the GPU, so the marshalling keeps its own share small: tensors by
# empty_like (the cheapest allocation call), raw addresses, and the raw stream without a Stream object around it.
_CONTIGUOUS = torch.contiguous_format
_empty_like = torch.empty_like
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _code(t, name):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)") from None


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t


def _need(t, name, device, dtype, shape, contiguous=True):
    """Checks an optional tensor (None passes) and returns its address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _addr(t):
    return None if t is None else t.data_ptr()


def _call(name, device, *args):
    """Calls an entry point with `device` current, and raises on a status other than KDA_OK."""
    fn = getattr(_lib.load(), name)
    if _current_device() == device.index:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st:
        check(name, st)


def _workspace(entry, device, args, given):
    """The workspace of a call: the given tensor, or one allocated for the size the query answers."""
    n = ctypes.c_size_t(0)
    _call(entry + "_workspace_size", device, ctypes.byref(args), ctypes.byref(n))
    if not n.value:
        return None
    ws = given if given is not None else torch.empty(n.value, dtype=torch.uint8, device=device)
    args.workspace = _need(ws, "workspace", device, torch.uint8, ws.shape)
    args.workspace_bytes = ws.numel()
    return ws


# ---------------------------------------------------------------- norms of queries and keys
def _token_strides(t, name):
    """(B, S, H, D) of a (B, S, H, D) or (S, H, D) tensor and its token strides; heads and channels contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 4:
        (B, S, H, D), (b, s, h, d) = shape, stride
    elif len(shape) == 3:
        (S, H, D), (s, h, d), B, b = shape, stride, 1, 0
    else:
        raise ValueError(f"{name} must have shape (B, S, H, D) or (S, H, D) (got {tuple(shape)})")
    if (d != 1 and D > 1) or (h != D and H > 1):
        raise ValueError(f"{name}: the heads and channels of a token must be contiguous")
    return B, S, H, D, (b if B > 1 else 0), (s if S > 1 else 0)


def _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved):
    dev, dt = _cuda(q, "q").device, q.dtype
    code = _code(q, "q")
    B, S, Hq, D, qb, qs = _token_strides(q, "q")
    if not isinstance(k, torch.Tensor) or k.device != dev:
        raise ValueError(f"k must be a tensor on {dev}")
    if k.dtype != dt:
        raise TypeError(f"k must be {dt} (got {k.dtype})")
    kB, kS, Hk, kD, kb, ks = _token_strides(k, "k")
    if kB != B or kS != S or kD != D or k.dim() != q.dim():
        raise ValueError(f"k's shape {tuple(k.shape)} does not go with q's {tuple(q.shape)}")
    qw = None if q_weight is None else _need(q_weight, "q_weight", dev, torch.float32, (D,))
    kw = None if k_weight is None else _need(k_weight, "k_weight", dev, torch.float32, (D,))
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    rot, pos, inv = 0, None, None
    if inv_freq is not None:
        n = inv_freq.numel()
        pos = _need(positions, "positions", dev, torch.int64, (B, S) if q.dim() == 4 else (S,))
        inv = _need(inv_freq, "inv_freq", dev, torch.float32, (n,))
        rot = 2 * n
    kind = NORMS.get(norm)
    if kind is None:
        raise ValueError(f"norm must be one of {sorted(NORMS)} (got {norm!r})")
    return QkNormArgs(B, S, Hq, Hk, D, code, q.data_ptr(), k.data_ptr(), qb, qs, kb, ks, kind, eps, qw, kw, pos, inv, rot,
                      bool(interleaved), None, None, _raw_stream(dev.index))


def qk_norm(q, k, *, norm="l2", eps=1e-6, q_weight=None, k_weight=None, positions=None, inv_freq=None,
            interleaved=False, out_q=None, out_k=None):
    """Per-head norm of queries and keys, and the rotation by position, in one pass (kda_qk_norm_fwd).

    q (B,S,H_q,D) and k (B,S,H_k,D), or without B; the heads of a token are
    contiguous, tokens may be strided (slices of a fused projection's rows).
    ``norm``: "l2" (x / sqrt(sum x^2 + eps)) or "rms" (mean instead of sum);
    ``q_weight`` / ``k_weight`` (D,) fp32 or None.  With ``inv_freq`` (R/2,)
    fp32 and ``positions`` (B,S) int64 the first R channels are rotated by
    position * inv_freq, in pairs (j, j + R/2) or, ``interleaved``, (2j, 2j + 1).
    Returns contiguous (q_out, k_out) in the inputs' dtype."""
    a = _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved)
    dev = q.device
    if out_q is None:
        out_q = _empty_like(q, memory_format=_CONTIGUOUS)
    if out_k is None:
        out_k = _empty_like(k, memory_format=_CONTIGUOUS)
    a.q_out = _need(out_q, "out_q", dev, q.dtype, q.shape)
    a.k_out = _need(out_k, "out_k", dev, q.dtype, k.shape)
    _call("kda_qk_norm_fwd", dev, ctypes.byref(a))
    return out_q, out_k


def qk_norm_bwd(q, k, dq_out, dk_out, *, norm="l2", eps=1e-6, q_weight=None, k_weight=None, positions=None,
                inv_freq=None, interleaved=False, workspace=None):
    """Gradients of ``qk_norm`` (kda_qk_norm_bwd): the forward's arguments, and dq_out, dk_out = dL/d(outputs), both
    fp32 or both in the inputs' dtype.  Returns a dict of dq, dk (inputs' dtype, contiguous) and dq_weight, dk_weight
    (fp32, None without that weight)."""
    f = _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved)
    dev = q.device
    gt = _cuda(dq_out, "dq_out").dtype
    if gt not in (torch.float32, q.dtype):
        raise TypeError(f"dq_out must be float32 or {q.dtype} (got {gt})")
    out = {"dq": _empty_like(q, memory_format=_CONTIGUOUS), "dk": _empty_like(k, memory_format=_CONTIGUOUS),
           "dq_weight": None if q_weight is None else _empty_like(q_weight),
           "dk_weight": None if k_weight is None else _empty_like(k_weight)}
    a = QkNormBwdArgs(f, _DT[gt], _need(dq_out, "dq_out", dev, gt, q.shape), _need(dk_out, "dk_out", dev, gt, k.shape),
                      out["dq"].data_ptr(), out["dk"].data_ptr(), _addr(out["dq_weight"]), _addr(out["dk_weight"]), None, 0)
    ws = _workspace("kda_qk_norm_bwd", dev, a, workspace)  # noqa: F841 (alive until the call has been queued)
    _call("kda_qk_norm_bwd", dev, ctypes.byref(a))
    return out


# ---------------------------------------------------------------- the gated delta rule
def gdn_decode_step(q, k, v, beta, state, *, z=None, log_decay=None, g_min=-5.0, gate_logits=None, eps=1e-6,
                    slots=None, out=None, dev_status=None):
    """The gated delta rule (one scalar decay per token and head) token by token (kda_gdn_decode_step).

    One token for B sequences: q, k (B,H,D_k); v, gate_logits (B,H,D_v); beta and
    z or log_decay (B,H).  T tokens each: the same with (B,T,H,...).  ``state``
    (num_slots,H,D_k,D_v) fp32 is advanced IN PLACE; ``slots`` (B,) int32 picks
    each sequence's state (None: the first B).  A negative slot is a padded row,
    whose rows of ``out`` stay as they were (unspecified when ``out`` is not given);
    a slot outside the pool, or given twice, is skipped like it and sets
    ``dev_status`` (a zeroed int32 tensor).  Returns o in the input dtype."""
    dev, dt = _cuda(q, "q").device, q.dtype
    code = _code(q, "q")
    if q.dim() not in (3, 4):
        raise ValueError(f"q must have shape (B, H, D_k) or (B, T, H, D_k) (got {tuple(q.shape)})")
    lead, Dk, Dv = q.shape[:-1], q.shape[-1], v.shape[-1]
    B, T, H = (lead[0], 1, lead[1]) if q.dim() == 3 else lead
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    vec = (*lead, Dv)
    if beta.dim() == len(lead) + 1 and beta.shape[-1] == 1:
        beta = beta.view(lead)
    if out is None:
        out = _empty_like(v)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must have shape (num_slots, H, D_k, D_v)")
    n = state.shape[0]
    a = GdnDecodeArgs(B, n, T, H, Dk, Dv, code, q.data_ptr(), _need(k, "k", dev, dt, q.shape), _need(v, "v", dev, dt, vec),
                      _need(z, "z", dev, dt, lead), _need(log_decay, "log_decay", dev, torch.float32, lead), g_min,
                      _need(beta, "beta", dev, dt, lead), _need(state, "state", dev, torch.float32, (n, H, Dk, Dv)),
                      _need(slots, "slots", dev, torch.int32, (B,)), _need(gate_logits, "gate_logits", dev, dt, vec), eps,
                      _need(out, "out", dev, dt, vec),
                      None if dev_status is None else _need(dev_status, "dev_status", dev, torch.int32, dev_status.shape),
                      _raw_stream(dev.index))
    _call("kda_gdn_decode_step", dev, ctypes.byref(a))
    return out


def gdn_chunk_bwd(q, k, v, beta, d_o, *, z=None, log_decay=None, g_min=-5.0, initial_state=None, d_final_state=None,
                  want_d_initial_state=True, workspace=None):
    """Gradients of the gated delta rule (kda_gdn_chunk_bwd), the core output o~ of ``gdn_chunk_fwd``: given d_o = dL/do~
    (B,S,H,D_v) and d_final_state = dL/dS_T (B,H,D_k,D_v) or None, a dict of fp32 tensors dq, dk (B,S,H,D_k), dv
    (B,S,H,D_v), dbeta and dz (or dlog_decay) (B,S,H), d_initial_state (or None).  z / log_decay: (B,S,H)."""
    dev, dt = _cuda(q, "q").device, q.dtype
    code = _code(q, "q")
    B, S, H, Dk = q.shape
    Dv = v.shape[-1]
    if beta.dim() == 4 and beta.shape[-1] == 1:
        beta = beta.view(B, S, H)
    tok, val, st, f32 = (B, S, H), (B, S, H, Dv), (B, H, Dk, Dv), torch.float32
    addr = {n: _need(t, n, dev, dt, shape) for n, t, shape in (("q", q, q.shape), ("k", k, q.shape), ("v", v, val),
                                                              ("z", z, tok), ("beta", beta, tok), ("d_o", d_o, val))}
    out = {"dq": _empty_like(q, dtype=f32), "dk": _empty_like(k, dtype=f32), "dv": _empty_like(v, dtype=f32),
           "dbeta": _empty_like(beta, dtype=f32), "dz": _empty_like(beta, dtype=f32),
           "d_initial_state": torch.empty(st, dtype=f32, device=dev) if want_d_initial_state else None}
    a = RecBwdArgs(B, S, H, Dk, Dv, code, addr["q"], addr["k"], addr["v"], addr["z"],
                   _need(log_decay, "log_decay", dev, f32, tok), g_min, addr["beta"],
                   _need(initial_state, "initial_state", dev, f32, st), addr["d_o"],
                   _need(d_final_state, "d_final_state", dev, f32, st), out["dq"].data_ptr(), out["dk"].data_ptr(),
                   out["dv"].data_ptr(), out["dbeta"].data_ptr(), out["dz"].data_ptr(), _addr(out["d_initial_state"]),
                   None, 0, _raw_stream(dev.index))
    ws = _workspace("kda_gdn_chunk_bwd", dev, a, workspace)  # noqa: F841 (alive until the call has been queued)
    _call("kda_gdn_chunk_bwd", dev, ctypes.byref(a))
    if log_decay is not None:
        out["dlog_decay"] = out.pop("dz")
    return out


# ---------------------------------------------------------------- the output path in e4m3
def quant_fp8(x, block_rows=1):
    """e4m3 values of a matrix x (..., K), float32 or bfloat16, and the fp32 scale of each block of 128 channels
    (kda_quant_fp8): block_rows = 1 for activations, 128 for weights (D_model, K).  Returns (x8, scales) with scales
    (..., ceil(K / 128)) or (ceil(D_model / 128), ceil(K / 128))."""
    dev = _cuda(x, "x").device
    code = _code(x, "x")
    _need(x, "x", dev, x.dtype, x.shape)
    if block_rows != 1 and x.dim() != 2:
        raise ValueError("blocks of several rows need a matrix")
    K = x.shape[-1]
    kb = -(-K // 128)
    rows = x.numel() // K if K else 0
    x8 = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
    shape = (*x.shape[:-1], kb) if block_rows == 1 else (-(-rows // block_rows) if block_rows > 0 else 0, kb)
    scales = torch.empty(shape, dtype=torch.float32, device=dev)
    _call("kda_quant_fp8", dev, x.data_ptr(), code, rows, K, block_rows, x8.data_ptr(), scales.data_ptr(), _raw_stream(dev.index))
    return x8, scales


def norm_gate_fp8(o, gate_logits, eps=1e-6):
    """Per-head RMSNorm over D_v, sigmoid gate and quantisation to e4m3 in one pass (kda_norm_gate_fp8); o, gate_logits
    (..., H, D_v).  Returns (x8 (..., H * D_v), scales (..., ceil(H * D_v / 128))) for ``out_proj_fp8``."""
    dev = _cuda(o, "o").device
    code = _code(o, "o")
    po, pg = _need(o, "o", dev, o.dtype, o.shape), _need(gate_logits, "gate_logits", dev, o.dtype, o.shape)
    H, Dv = o.shape[-2:]
    lead, K = o.shape[:-2], H * Dv
    x8 = o.new_empty((*lead, K), dtype=torch.float8_e4m3fn)
    scales = o.new_empty((*lead, -(-K // 128)), dtype=torch.float32)
    N = o.numel() // K if K else 0
    _call("kda_norm_gate_fp8", dev, po, pg, N, H, Dv, eps, code, x8.data_ptr(), scales.data_ptr(),
          _raw_stream(dev.index))
    return x8, scales


def out_proj_fp8(x8, x_scale, W8, W_scale, out_dtype=torch.bfloat16, out=None):
    """y = x W_o^T from e4m3 operands with a scale per block of 128 (kda_out_proj_fp8): x8 (..., K) and x_scale
    (..., ceil(K / 128)); W8 (D_model, K) and W_scale (ceil(D_model / 128), ceil(K / 128)), as ``norm_gate_fp8`` and
    ``quant_fp8(W_o, 128)`` give them.  Returns y (..., D_model) in ``out_dtype``."""
    dev = _cuda(x8, "x8").device
    Dm, K = W8.shape
    kb = -(-K // 128)
    lead = x8.shape[:-1]
    px = _need(x8, "x8", dev, torch.float8_e4m3fn, (*lead, K))
    ps = _need(x_scale, "x_scale", dev, torch.float32, (*lead, kb))
    pw = _need(W8, "W8", dev, torch.float8_e4m3fn, (Dm, K))
    pv = _need(W_scale, "W_scale", dev, torch.float32, (-(-Dm // 128), kb))
    code = _DT.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
    if out is None:
        out = x_scale.new_empty((*lead, Dm), dtype=out_dtype)
    py = _need(out, "out", dev, out_dtype, (*lead, Dm))
    N = x8.numel() // K if K else 0
    _call("kda_out_proj_fp8", dev, px, ps, pw, pv, N, K, Dm, py, code, _raw_stream(dev.index))
    return out

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
# empty_like (the cheapest allocation call), one test per tensor on the way that passes, packed arguments, and the raw
# stream without a Stream object around it.
_CONTIGUOUS = torch.contiguous_format
_empty_like = torch.empty_like
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_F32 = torch.float32
_pack_qk_norm = _lib.packer(QkNormArgs).pack
_pack_gdn_decode = _lib.packer(GdnDecodeArgs).pack


def _start(t, name):
    """Device index and dtype code of the call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _DT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    return t.get_device(), code


def _need(t, name, index, dtype, shape):
    """The address of a tensor of the call (0 for None), which must be as described.  (The calls of single tokens make the
    same test in place, and come here when it fails.)"""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise ValueError(f"{name} must be a tensor on cuda:{index}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_entry = {}  # the library's functions by name, as they are first called


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _call(name, index, *args):
    """Calls an entry point with device `index` current, and raises on a status other than KDA_OK."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(_lib.load(), name)
    if _current_device() == index:
        st = fn(*args)
    else:
        with torch.cuda.device(index):
            st = fn(*args)
    if st:
        check(name, st)


def _workspace(entry, index, args, given):
    """The workspace of a call: the given tensor, or one allocated for the size the query answers."""
    n = ctypes.c_size_t(0)
    _call(entry + "_workspace_size", index, ctypes.byref(args), ctypes.byref(n))
    if not n.value:
        return None
    ws = given if given is not None else torch.empty(n.value, dtype=torch.uint8, device=torch.device("cuda", index))
    args.workspace = _need(ws, "workspace", index, torch.uint8, getattr(ws, "shape", None))
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
    """(device index, the fields of QkNormArgs before its outputs)."""
    ix, code = _start(q, "q")
    B, S, Hq, D, qb, qs = _token_strides(q, "q")
    if not isinstance(k, torch.Tensor) or k.get_device() != ix:
        raise ValueError(f"k must be a tensor on cuda:{ix}")
    if k.dtype is not q.dtype:
        raise TypeError(f"k must be {q.dtype} (got {k.dtype})")
    kB, kS, Hk, kD, kb, ks = _token_strides(k, "k")
    if kB != B or kS != S or kD != D or k.dim() != q.dim():
        raise ValueError(f"k's shape {tuple(k.shape)} does not go with q's {tuple(q.shape)}")
    rot = pos = inv = 0
    if inv_freq is not None:
        if positions is None:
            raise ValueError("positions and inv_freq go together")
        n = inv_freq.numel()
        if (positions.dtype is not torch.int64 or positions.shape != q.shape[:-2] or positions.get_device() != ix or
                not positions.is_contiguous()):
            _need(positions, "positions", ix, torch.int64, q.shape[:-2])
        pos, inv, rot = positions.data_ptr(), _need(inv_freq, "inv_freq", ix, _F32, (n,)), 2 * n
    elif positions is not None:
        raise ValueError("positions and inv_freq go together")
    kind = NORMS.get(norm)
    if kind is None:
        raise ValueError(f"norm must be one of {sorted(NORMS)} (got {norm!r})")
    qw = kw = 0
    if q_weight is not None:
        qw = _need(q_weight, "q_weight", ix, _F32, (D,))
    if k_weight is not None:
        kw = _need(k_weight, "k_weight", ix, _F32, (D,))
    return ix, (B, S, Hq, Hk, D, code, q.data_ptr(), k.data_ptr(), qb, qs, kb, ks, kind, eps, qw, kw, pos, inv, rot,
                1 if interleaved else 0)


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
    ix, a = _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved)
    if out_q is None:
        out_q = _empty_like(q, memory_format=_CONTIGUOUS)
        oq = out_q.data_ptr()
    else:
        oq = _need(out_q, "out_q", ix, q.dtype, q.shape)
    if out_k is None:
        out_k = _empty_like(k, memory_format=_CONTIGUOUS)
        ok = out_k.data_ptr()
    else:
        ok = _need(out_k, "out_k", ix, q.dtype, k.shape)
    _call("kda_qk_norm_fwd", ix, _pack_qk_norm(*a, oq, ok, _raw_stream(ix)))
    return out_q, out_k


def qk_norm_bwd(q, k, dq_out, dk_out, *, norm="l2", eps=1e-6, q_weight=None, k_weight=None, positions=None,
                inv_freq=None, interleaved=False, workspace=None):
    """Gradients of ``qk_norm`` (kda_qk_norm_bwd): the forward's arguments, and dq_out, dk_out = dL/d(outputs), both
    fp32 or both in the inputs' dtype.  Returns a dict of dq, dk (inputs' dtype, contiguous) and dq_weight, dk_weight
    (fp32, None without that weight)."""
    ix, f = _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved)
    gt = getattr(dq_out, "dtype", None)
    if gt not in (_F32, q.dtype):
        raise TypeError(f"dq_out must be float32 or {q.dtype} (got {gt})")
    out = {"dq": _empty_like(q, memory_format=_CONTIGUOUS), "dk": _empty_like(k, memory_format=_CONTIGUOUS),
           "dq_weight": None if q_weight is None else _empty_like(q_weight),
           "dk_weight": None if k_weight is None else _empty_like(k_weight)}
    a = QkNormBwdArgs(QkNormArgs(*f, 0, 0, _raw_stream(ix)), _DT[gt], _need(dq_out, "dq_out", ix, gt, q.shape),
                      _need(dk_out, "dk_out", ix, gt, k.shape), out["dq"].data_ptr(), out["dk"].data_ptr(),
                      _addr(out["dq_weight"]), _addr(out["dk_weight"]), 0, 0)
    ws = _workspace("kda_qk_norm_bwd", ix, a, workspace)  # noqa: F841 (alive until the call has been queued)
    _call("kda_qk_norm_bwd", ix, ctypes.byref(a))
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
    ix, code = _start(q, "q")
    dt, shape = q.dtype, q.shape
    if len(shape) == 3:
        (B, H, Dk), T, tok = shape, 1, shape[:2]
    elif len(shape) == 4:
        (B, T, H, Dk), tok = shape, shape[:3]
    else:
        raise ValueError(f"q must have shape (B, H, D_k) or (B, T, H, D_k) (got {tuple(shape)})")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    Dv = v.shape[-1]
    val = (*tok, Dv)
    if k.dtype is not dt or k.shape != shape or k.get_device() != ix or not k.is_contiguous():
        _need(k, "k", ix, dt, shape)
    if v.dtype is not dt or v.shape != val or v.get_device() != ix or not v.is_contiguous():
        _need(v, "v", ix, dt, val)
    if beta.dtype is not dt or beta.shape != tok or beta.get_device() != ix or not beta.is_contiguous():
        if beta.dim() == len(tok) + 1 and beta.shape[-1] == 1:
            beta = beta.view(tok)
        _need(beta, "beta", ix, dt, tok)
    n = state.shape[0]
    if (state.dtype is not _F32 or state.shape != (n, H, Dk, Dv) or state.get_device() != ix or
            not state.is_contiguous()):
        _need(state, "state", ix, _F32, (n, H, Dk, Dv))
    pz = pl = ps = pg = pd = 0
    if z is not None:
        pz = _need(z, "z", ix, dt, tok)
    if log_decay is not None:
        pl = _need(log_decay, "log_decay", ix, _F32, tok)
    if slots is not None:
        ps = _need(slots, "slots", ix, torch.int32, (B,))
    if gate_logits is not None:
        pg = _need(gate_logits, "gate_logits", ix, dt, val)
    if dev_status is not None:
        pd = _need(dev_status, "dev_status", ix, torch.int32, dev_status.shape)
    if out is None:
        out = _empty_like(v)
    else:
        _need(out, "out", ix, dt, val)
    _call("kda_gdn_decode_step", ix, _pack_gdn_decode(
        B, n, T, H, Dk, Dv, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), pz, pl, g_min, beta.data_ptr(),
        state.data_ptr(), ps, pg, eps, out.data_ptr(), pd, _raw_stream(ix)))
    return out


def gdn_chunk_bwd(q, k, v, beta, d_o, *, z=None, log_decay=None, g_min=-5.0, initial_state=None, d_final_state=None,
                  want_d_initial_state=True, workspace=None):
    """Gradients of the gated delta rule (kda_gdn_chunk_bwd), the core output o~ of ``gdn_chunk_fwd``: given d_o = dL/do~
    (B,S,H,D_v) and d_final_state = dL/dS_T (B,H,D_k,D_v) or None, a dict of fp32 tensors dq, dk (B,S,H,D_k), dv
    (B,S,H,D_v), dbeta and dz (or dlog_decay) (B,S,H), d_initial_state (or None).  z / log_decay: (B,S,H)."""
    ix, code = _start(q, "q")
    dt = q.dtype
    B, S, H, Dk = q.shape
    Dv = v.shape[-1]
    if beta.dim() == 4 and beta.shape[-1] == 1:
        beta = beta.view(B, S, H)
    tok, val, st = (B, S, H), (B, S, H, Dv), (B, H, Dk, Dv)
    addr = {n: _need(t, n, ix, dt, shape) for n, t, shape in (("q", q, q.shape), ("k", k, q.shape), ("v", v, val),
                                                             ("z", z, tok), ("beta", beta, tok), ("d_o", d_o, val))}
    out = {"dq": _empty_like(q, dtype=_F32), "dk": _empty_like(k, dtype=_F32), "dv": _empty_like(v, dtype=_F32),
           "dbeta": _empty_like(beta, dtype=_F32), "dz": _empty_like(beta, dtype=_F32),
           "d_initial_state": q.new_empty(st, dtype=_F32) if want_d_initial_state else None}
    a = RecBwdArgs(B, S, H, Dk, Dv, code, addr["q"], addr["k"], addr["v"], addr["z"],
                   _need(log_decay, "log_decay", ix, _F32, tok), g_min, addr["beta"],
                   _need(initial_state, "initial_state", ix, _F32, st), addr["d_o"],
                   _need(d_final_state, "d_final_state", ix, _F32, st), out["dq"].data_ptr(), out["dk"].data_ptr(),
                   out["dv"].data_ptr(), out["dbeta"].data_ptr(), out["dz"].data_ptr(), _addr(out["d_initial_state"]),
                   0, 0, _raw_stream(ix))
    ws = _workspace("kda_gdn_chunk_bwd", ix, a, workspace)  # noqa: F841 (alive until the call has been queued)
    _call("kda_gdn_chunk_bwd", ix, ctypes.byref(a))
    if log_decay is not None:
        out["dlog_decay"] = out.pop("dz")
    return out


# ---------------------------------------------------------------- the output path in e4m3
def quant_fp8(x, block_rows=1):
    """e4m3 values of a matrix x (..., K), float32 or bfloat16, and the fp32 scale of each block of 128 channels
    (kda_quant_fp8): block_rows = 1 for activations, 128 for weights (D_model, K).  Returns (x8, scales) with scales
    (..., ceil(K / 128)) or (ceil(D_model / 128), ceil(K / 128))."""
    ix, code = _start(x, "x")
    px = _need(x, "x", ix, x.dtype, x.shape)
    if block_rows != 1 and x.dim() != 2:
        raise ValueError("blocks of several rows need a matrix")
    K = x.shape[-1]
    kb = -(-K // 128)
    rows = x.numel() // K if K else 0
    x8 = _empty_like(x, dtype=torch.float8_e4m3fn)
    shape = (*x.shape[:-1], kb) if block_rows == 1 else (-(-rows // block_rows) if block_rows > 0 else 0, kb)
    scales = x.new_empty(shape, dtype=_F32)
    _call("kda_quant_fp8", ix, px, code, rows, K, block_rows, x8.data_ptr(), scales.data_ptr(), _raw_stream(ix))
    return x8, scales


def norm_gate_fp8(o, gate_logits, eps=1e-6):
    """Per-head RMSNorm over D_v, sigmoid gate and quantisation to e4m3 in one pass (kda_norm_gate_fp8); o, gate_logits
    (..., H, D_v).  Returns (x8 (..., H * D_v), scales (..., ceil(H * D_v / 128))) for ``out_proj_fp8``."""
    ix, code = _start(o, "o")
    shape = o.shape
    po, pg = _need(o, "o", ix, o.dtype, shape), _need(gate_logits, "gate_logits", ix, o.dtype, shape)
    H, Dv = shape[-2:]
    lead, K = shape[:-2], H * Dv
    x8 = o.new_empty((*lead, K), dtype=torch.float8_e4m3fn)
    scales = o.new_empty((*lead, -(-K // 128)), dtype=_F32)
    _call("kda_norm_gate_fp8", ix, po, pg, o.numel() // K if K else 0, H, Dv, eps, code, x8.data_ptr(),
          scales.data_ptr(), _raw_stream(ix))
    return x8, scales


def out_proj_fp8(x8, x_scale, W8, W_scale, out_dtype=torch.bfloat16, out=None):
    """y = x W_o^T from e4m3 operands with a scale per block of 128 (kda_out_proj_fp8): x8 (..., K) and x_scale
    (..., ceil(K / 128)); W8 (D_model, K) and W_scale (ceil(D_model / 128), ceil(K / 128)), as ``norm_gate_fp8`` and
    ``quant_fp8(W_o, 128)`` give them.  Returns y (..., D_model) in ``out_dtype``."""
    if not isinstance(x8, torch.Tensor) or not x8.is_cuda:
        raise ValueError("x8 must be a CUDA tensor")
    ix = x8.get_device()
    Dm, K = W8.shape
    kb = -(-K // 128)
    lead = x8.shape[:-1]
    px = _need(x8, "x8", ix, torch.float8_e4m3fn, (*lead, K))
    ps = _need(x_scale, "x_scale", ix, _F32, (*lead, kb))
    pw = _need(W8, "W8", ix, torch.float8_e4m3fn, (Dm, K))
    pv = _need(W_scale, "W_scale", ix, _F32, (-(-Dm // 128), kb))
    code = _DT.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
    if out is None:
        out = x_scale.new_empty((*lead, Dm), dtype=out_dtype)
        py = out.data_ptr()
    else:
        py = _need(out, "out", ix, out_dtype, (*lead, Dm))
    _call("kda_out_proj_fp8", ix, px, ps, pw, pv, x8.numel() // K if K else 0, K, Dm, py, code, _raw_stream(ix))
    return out

"""Torch-facing entry points of the operators around the gated delta rule.

The norm of queries and keys with the rotation by position and its gradients;
the gated delta rule token by token and its gradients; the output path in e4m3.
Every step runs inside libkda's CUDA kernels, on the current stream of the
tensors' device (which need not be the current device).  Checks, allocation and
the call itself are in csrc_py/marshal.cpp: these calls can take a few
microseconds on the GPU, and marshalling their arguments in Python took longer.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import check
from .api import _DT

NORMS = {"l2": _lib.NORM_L2, "rms": _lib.NORM_RMS}


def _bind():
    """Hands the loaded library's entry points to the marshalling."""
    lib = _lib.load()
    _m.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _lib.SIGNATURES})


class _Unloaded:
    """Stands for the extension until its first use: the package imports without it, since the build runs from here."""

    def __getattr__(self, name):
        global _m
        try:
            from . import _marshal
        except ImportError as e:
            raise ImportError("_marshal.so is missing or does not fit this torch: build it with `python -m "
                              "kimi_delta_attention_21_b200.build` (there is no other path)") from e
        _marshal.loader(_bind)
        _m = _marshal
        return getattr(_marshal, name)


_m = _Unloaded()


def _done(name, result):
    """The results of a call, or the error behind its status."""
    if result.__class__ is int:
        check(name, result)
    return result


def _norm(kind):
    try:
        return NORMS[kind]
    except KeyError:
        raise ValueError(f"norm must be one of {sorted(NORMS)} (got {kind!r})") from None


# ---------------------------------------------------------------- norms of queries and keys
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
    return _done("kda_qk_norm_fwd", _m.qk_norm(q, k, _norm(norm), eps, q_weight, k_weight, positions, inv_freq, interleaved,
                                               out_q, out_k))


def qk_norm_bwd(q, k, dq_out, dk_out, *, norm="l2", eps=1e-6, q_weight=None, k_weight=None, positions=None,
                inv_freq=None, interleaved=False, workspace=None):
    """Gradients of ``qk_norm`` (kda_qk_norm_bwd): the forward's arguments, and dq_out, dk_out = dL/d(outputs), both
    fp32 or both in the inputs' dtype.  Returns a dict of dq, dk (inputs' dtype, contiguous) and dq_weight, dk_weight
    (fp32, None without that weight)."""
    r = _done("kda_qk_norm_bwd", _m.qk_norm_bwd(q, k, _norm(norm), eps, q_weight, k_weight, positions, inv_freq, interleaved,
                                                dq_out, dk_out, workspace))
    return dict(zip(("dq", "dk", "dq_weight", "dk_weight"), r))


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
    return _done("kda_gdn_decode_step", _m.gdn_decode_step(q, k, v, beta, state, z, log_decay, g_min, gate_logits, eps, slots,
                                                           out, dev_status))


def gdn_chunk_bwd(q, k, v, beta, d_o, *, z=None, log_decay=None, g_min=-5.0, initial_state=None, d_final_state=None,
                  want_d_initial_state=True, workspace=None):
    """Gradients of the gated delta rule (kda_gdn_chunk_bwd), the core output o~ of ``gdn_chunk_fwd``: given d_o = dL/do~
    (B,S,H,D_v) and d_final_state = dL/dS_T (B,H,D_k,D_v) or None, a dict of fp32 tensors dq, dk (B,S,H,D_k), dv
    (B,S,H,D_v), dbeta and dz (or dlog_decay) (B,S,H), d_initial_state (or None).  z / log_decay: (B,S,H)."""
    r = _done("kda_gdn_chunk_bwd", _m.gdn_chunk_bwd(q, k, v, beta, d_o, z, log_decay, g_min, initial_state, d_final_state,
                                                    want_d_initial_state, workspace))
    return dict(zip(("dq", "dk", "dv", "dbeta", "dz" if log_decay is None else "dlog_decay", "d_initial_state"), r))


# ---------------------------------------------------------------- the output path in e4m3
def quant_fp8(x, block_rows=1):
    """e4m3 values of a matrix x (..., K), float32 or bfloat16, and the fp32 scale of each block of 128 channels
    (kda_quant_fp8): block_rows = 1 for activations, 128 for weights (D_model, K).  Returns (x8, scales) with scales
    (..., ceil(K / 128)) or (ceil(D_model / 128), ceil(K / 128))."""
    return _done("kda_quant_fp8", _m.quant_fp8(x, block_rows))


def norm_gate_fp8(o, gate_logits, eps=1e-6):
    """Per-head RMSNorm over D_v, sigmoid gate and quantisation to e4m3 in one pass (kda_norm_gate_fp8); o, gate_logits
    (..., H, D_v).  Returns (x8 (..., H * D_v), scales (..., ceil(H * D_v / 128))) for ``out_proj_fp8``."""
    return _done("kda_norm_gate_fp8", _m.norm_gate_fp8(o, gate_logits, eps))


def out_proj_fp8(x8, x_scale, W8, W_scale, out_dtype=torch.bfloat16, out=None):
    """y = x W_o^T from e4m3 operands with a scale per block of 128 (kda_out_proj_fp8): x8 (..., K) and x_scale
    (..., ceil(K / 128)); W8 (D_model, K) and W_scale (ceil(D_model / 128), ceil(K / 128)), as ``norm_gate_fp8`` and
    ``quant_fp8(W_o, 128)`` give them.  Returns y (..., D_model) in ``out_dtype``."""
    code = _DT.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be float32 or bfloat16 (got {out_dtype})")
    return _done("kda_out_proj_fp8", _m.out_proj_fp8(x8, x_scale, W8, W_scale, code, out))

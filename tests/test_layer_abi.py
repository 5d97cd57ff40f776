"""Host side of the operators around the gated delta rule: their structs match
the header, and bad calls are refused before anything is launched (fake device
addresses, never dereferenced)."""
import ctypes
import os
import subprocess

import pytest
import torch

import kimi_delta_attention_21_b200 as K
from kimi_delta_attention_21_b200 import _lib as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kda.h")
G = 1 << 30
P = [(1 << 40) + i * G for i in range(24)]  # one GiB apart

STRUCTS = {"kda_qk_norm_args": L.QkNormArgs, "kda_qk_norm_bwd_args": L.QkNormBwdArgs,
           "kda_gdn_decode_args": L.GdnDecodeArgs}


def test_struct_layouts_match_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    for c, S in STRUCTS.items():
        lines.append(f'printf("{c} sizeof %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in S._fields_]
    prog, exe = tmp_path / "layout.c", tmp_path / "layout"
    prog.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.check_call(["gcc", "-std=c11", "-o", str(exe), str(prog)])
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        c, f, n = line.split()
        S = STRUCTS[c]
        assert int(n) == (ctypes.sizeof(S) if f == "sizeof" else getattr(S, f).offset), (c, f)


def refused(fn, args, status, *more):
    lib = L.load()
    n0 = lib.kda_launch_count()
    assert getattr(lib, fn)(ctypes.byref(args), *more) == status, lib.kda_last_error().decode()
    assert lib.kda_last_error().decode() != ""
    assert lib.kda_launch_count() == n0


def qk(**kw):
    a = dict(B=2, S=8, H_q=4, H_k=2, D=64, dtype=L.KDA_BF16, q=P[0], k=P[1], q_stride_b=2048, q_stride_s=256,
             k_stride_b=1024, k_stride_s=128, norm=L.NORM_RMS, eps=1e-6, positions=P[4], inv_freq=P[5], rot_dim=64,
             q_out=P[2], k_out=P[3])
    a.update(kw)
    return L.QkNormArgs(**a)


@pytest.mark.parametrize("mut,status", [
    (dict(dtype=5), L.KDA_ERR_UNSUPPORTED), (dict(B=-1), L.KDA_ERR_INVALID_ARG), (dict(H_k=0), L.KDA_ERR_INVALID_ARG),
    (dict(D=257), L.KDA_ERR_UNSUPPORTED), (dict(rot_dim=63), L.KDA_ERR_INVALID_ARG),
    (dict(rot_dim=66), L.KDA_ERR_INVALID_ARG), (dict(norm=2), L.KDA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), L.KDA_ERR_INVALID_ARG), (dict(q=None), L.KDA_ERR_INVALID_ARG),
    (dict(k=P[1] + 1), L.KDA_ERR_INVALID_ARG), (dict(positions=None), L.KDA_ERR_INVALID_ARG),
    (dict(inv_freq=None), L.KDA_ERR_INVALID_ARG), (dict(q_out=None), L.KDA_ERR_INVALID_ARG),
    (dict(q_out=P[1] + 64), L.KDA_ERR_INVALID_ARG), (dict(k_out=P[2] + 128), L.KDA_ERR_INVALID_ARG),
    (dict(q_stride_s=-1), L.KDA_ERR_INVALID_ARG), (dict(k_stride_b=1 << 41), L.KDA_ERR_INVALID_ARG),
    (dict(B=1 << 20, S=1 << 20), L.KDA_ERR_UNSUPPORTED), (dict(H_q=1 << 20), L.KDA_ERR_UNSUPPORTED),
    (dict(q_weight=P[6] + 2), L.KDA_ERR_INVALID_ARG),
])
def test_qk_norm_refusals(mut, status):
    refused("kda_qk_norm_fwd", qk(**mut), status)


def test_qk_norm_bwd_refusals():
    def args(fwd=None, **kw):
        a = dict(fwd=fwd or qk(), grad_dtype=L.KDA_F32, dq_out=P[7], dk_out=P[8], dq=P[9], dk=P[10], dq_weight=P[11],
                 workspace=P[12], workspace_bytes=1 << 28)
        a.update(kw)
        return L.QkNormBwdArgs(**a)

    bad, unsup = L.KDA_ERR_INVALID_ARG, L.KDA_ERR_UNSUPPORTED
    refused("kda_qk_norm_bwd", args(grad_dtype=3), unsup)
    refused("kda_qk_norm_bwd", args(fwd=qk(dtype=L.KDA_F32), grad_dtype=L.KDA_BF16), unsup)
    refused("kda_qk_norm_bwd", args(workspace=None), L.KDA_ERR_WORKSPACE)
    refused("kda_qk_norm_bwd", args(workspace_bytes=64), L.KDA_ERR_WORKSPACE)
    refused("kda_qk_norm_bwd", args(dq_out=None), bad)
    refused("kda_qk_norm_bwd", args(dq=P[0]), bad)              # over an input
    refused("kda_qk_norm_bwd", args(dk=P[9] + 64), bad)         # over another output
    refused("kda_qk_norm_bwd", args(workspace=P[11]), bad)      # over a weight's gradient
    n = ctypes.c_size_t(7)
    a = args(dq_weight=None)
    assert L.load().kda_qk_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == L.KDA_OK and n.value == 0


@pytest.mark.parametrize("mut,status", [
    (dict(dtype=2), L.KDA_ERR_UNSUPPORTED), (dict(g_min=0.0), L.KDA_ERR_INVALID_ARG), (dict(T=-1), L.KDA_ERR_INVALID_ARG),
    (dict(D_v=129), L.KDA_ERR_UNSUPPORTED), (dict(B=1 << 31), L.KDA_ERR_UNSUPPORTED),
    (dict(num_slots=-1), L.KDA_ERR_INVALID_ARG), (dict(num_slots=3), L.KDA_ERR_INVALID_ARG),  # 4 sequences, no slots
    (dict(num_slots=1 << 41), L.KDA_ERR_UNSUPPORTED), (dict(k=None), L.KDA_ERR_INVALID_ARG),
    (dict(z=None), L.KDA_ERR_INVALID_ARG), (dict(state=None), L.KDA_ERR_INVALID_ARG),
    (dict(state=P[5] + 2), L.KDA_ERR_INVALID_ARG), (dict(slots=P[7] + 1), L.KDA_ERR_INVALID_ARG),
    (dict(o=P[2] + 64), L.KDA_ERR_INVALID_ARG), (dict(o=P[5] + 64), L.KDA_ERR_INVALID_ARG),
    (dict(state=P[0]), L.KDA_ERR_INVALID_ARG), (dict(gate_logits=P[8], eps=-1.0), L.KDA_ERR_INVALID_ARG),
])
def test_gdn_decode_refusals(mut, status):
    a = dict(B=4, num_slots=4, T=2, H=3, D_k=32, D_v=32, dtype=L.KDA_BF16, q=P[0], k=P[1], v=P[2], z=P[3], g_min=-5.0,
             beta=P[4], state=P[5], o=P[6], eps=1e-6)
    a.update(mut)
    refused("kda_gdn_decode_step", L.GdnDecodeArgs(**a), status)


def call_refused(fn, status, *args):
    lib = L.load()
    n0 = lib.kda_launch_count()
    assert getattr(lib, fn)(*args) == status, lib.kda_last_error().decode()
    assert lib.kda_launch_count() == n0


def test_fp8_refusals():
    bad, unsup, big = L.KDA_ERR_INVALID_ARG, L.KDA_ERR_UNSUPPORTED, 1 << 30
    q = lambda status, x=P[0], dt=1, r=4, c=256, br=1, x8=P[1], sc=P[2]: call_refused(
        "kda_quant_fp8", status, x, dt, r, c, br, x8, sc, None)
    q(unsup, dt=3)
    q(bad, r=-1)
    q(bad, c=0)
    q(bad, br=2)
    q(unsup, r=1 << 40, c=1 << 20)
    q(bad, x=None)
    q(bad, x=P[0] + 1)
    q(bad, x8=P[0] + 64)
    q(bad, sc=P[1] + 64)
    n = lambda status, o=P[0], g=P[1], N=4, H=2, Dv=128, eps=1e-6, dt=1, x8=P[2], sc=P[3]: call_refused(
        "kda_norm_gate_fp8", status, o, g, N, H, Dv, eps, dt, x8, sc, None)
    n(unsup, dt=9)
    n(bad, H=0)
    n(bad, eps=-1.0)
    n(unsup, H=8193)
    n(unsup, N=1 << 31)
    n(bad, g=None)
    n(bad, x8=P[1])
    n(bad, sc=P[2])
    p = lambda status, x=P[0], xs=P[1], w=P[2], ws=P[3], N=4, K=256, M=64, y=P[4], dt=1: call_refused(
        "kda_out_proj_fp8", status, x, xs, w, ws, N, K, M, y, dt, None)
    p(unsup, dt=2)
    p(bad, K=0)
    p(bad, N=-1)
    p(unsup, N=1 << 31)
    p(unsup, N=big, M=big)
    p(bad, xs=None)
    p(bad, ws=P[3] + 2)
    p(bad, y=P[0])
    p(bad, y=P[4] + 1)
    p(L.KDA_OK, N=0)


def gdn_bwd(**kw):
    a = dict(B=1, S=130, H=2, D_k=32, D_v=48, dtype=L.KDA_BF16, q=P[0], k=P[1], v=P[2], z=P[3], g_min=-5.0, beta=P[4],
             d_o=P[5], dq=P[6], dk=P[7], dv=P[8], dbeta=P[9], dz=P[10], workspace=P[11], workspace_bytes=1 << 29)
    a.update(kw)
    return L.RecBwdArgs(**a)


@pytest.mark.parametrize("mut,status", [
    (dict(dtype=4), L.KDA_ERR_UNSUPPORTED), (dict(g_min=0.5), L.KDA_ERR_INVALID_ARG), (dict(S=-1), L.KDA_ERR_INVALID_ARG),
    (dict(D_k=129), L.KDA_ERR_UNSUPPORTED), (dict(S=64 << 28, H=16), L.KDA_ERR_UNSUPPORTED),
    (dict(B=1 << 28, S=1, H=1), L.KDA_ERR_UNSUPPORTED), (dict(d_o=None), L.KDA_ERR_INVALID_ARG),
    (dict(z=None), L.KDA_ERR_INVALID_ARG), (dict(dz=None), L.KDA_ERR_INVALID_ARG),
    (dict(workspace_bytes=1000), L.KDA_ERR_WORKSPACE), (dict(workspace=None), L.KDA_ERR_WORKSPACE),
    (dict(workspace=P[11] + 16), L.KDA_ERR_INVALID_ARG), (dict(dq=P[0]), L.KDA_ERR_INVALID_ARG),
    (dict(dz=P[9] + 16), L.KDA_ERR_INVALID_ARG), (dict(d_initial_state=P[11] + 1024), L.KDA_ERR_INVALID_ARG),
])
def test_gdn_bwd_refusals(mut, status):
    refused("kda_gdn_chunk_bwd", gdn_bwd(**mut), status)


@pytest.mark.parametrize("B,S,H,Dk,Dv", [(1, 4096, 16, 128, 128), (2, 100, 3, 18, 13), (0, 5, 1, 8, 8), (2, 0, 1, 8, 8)])
def test_gdn_bwd_workspace_is_one_record_per_chunk(B, S, H, Dk, Dv):
    n, up = ctypes.c_size_t(1), lambda x, m: -(-x // m) * m
    a = gdn_bwd(B=B, S=S, H=H, D_k=Dk, D_v=Dv)
    assert L.load().kda_gdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == L.KDA_OK
    dk, dv = up(Dk, 16), up(Dv, 32)
    assert n.value == B * H * -(-S // 64) * 4 * (256 + 12288 + 64 * (dk + 2 * dv) + 2 * dk * dv)


Z = torch.zeros


@pytest.mark.parametrize("call,error,text", [
    (lambda: K.qk_norm(Z(2, 2, 2), Z(2, 2, 2)), ValueError, "q must be a CUDA tensor"),
    (lambda: K.qk_norm(None, Z(2, 2, 2)), ValueError, "q must be a CUDA tensor"),
    (lambda: K.qk_norm(Z(2, 2, 2), Z(2, 2, 2), norm="layer"), ValueError, "norm must be one of"),
    (lambda: K.qk_norm_bwd(*[Z(2, 2, 2)] * 4), ValueError, "q must be a CUDA tensor"),
    (lambda: K.gdn_decode_step(*[Z(2, 2, 2)] * 5, z=Z(2, 2)), ValueError, "q must be a CUDA tensor"),
    (lambda: K.gdn_chunk_bwd(*[Z(1, 1, 1, 1)] * 5), ValueError, "q must be a CUDA tensor"),
    (lambda: K.quant_fp8(Z(4, 4)), ValueError, "x must be a CUDA tensor"),
    (lambda: K.norm_gate_fp8(Z(2, 2), Z(2, 2)), ValueError, "o must be a CUDA tensor"),
    (lambda: K.out_proj_fp8(*[Z(2, 2)] * 4), ValueError, "x8 must be a CUDA tensor"),
    (lambda: K.out_proj_fp8(*[Z(2, 2)] * 4, out_dtype=torch.half), TypeError, "out_dtype"),
])
def test_python_calls_without_device_tensors_are_refused(call, error, text):
    n0 = L.load().kda_launch_count()
    with pytest.raises(error, match=text):
        call()
    assert L.load().kda_launch_count() == n0

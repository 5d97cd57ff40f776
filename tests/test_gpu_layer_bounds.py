"""The bounds-checked build over every way through the operators around the gated delta rule: no write outside its buffer,
the normal build's bits; and with every buffer said to be one byte shorter than it is, the last element of each output and
workspace is seen, skipped and counted (so the first test looks at something)."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import Guarded, gen, randn  # noqa: E402

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def child(out, *args, **env):
    r = subprocess.run([sys.executable, os.path.join(HERE, "layer_bounds_cases.py"), str(out), *args],
                       env=dict(os.environ, KDA_LIBRARY="libkda_checked.so", **env), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    return np.load(out)


def test_no_write_leaves_its_buffer(tmp_path):
    import layer_bounds_cases
    got = child(tmp_path / "all.npz")
    assert int(got["_checked"]) == 1 and int(got["_errors"]) == 0
    want, (errors, checked) = layer_bounds_cases.run_cases()
    assert (errors, checked) == (0, 0)
    assert set(want) == {n for n in got.files if not n.startswith("_")}
    for n, x in want.items():
        assert np.array_equal(got[n], x, equal_nan=True), f"{n}: checked and normal builds differ"


def test_the_last_element_of_every_output_is_checked(tmp_path):
    import layer_bounds_cases
    got = child(tmp_path / "last.npz", "last", KDA_CHECKED_SHRINK="1")
    assert set(got.files) == {n for n, _ in layer_bounds_cases.calls()}
    for n in got.files:
        skipped, written = got[n]
        assert int(skipped) > 0, f"{n}: no write is checked"
        assert written == "", f"{n}: written without a check: {written}"


@pytest.mark.parametrize("D,R,dtype,gdtype", [(128, 128, torch.bfloat16, torch.float32), (96, 0, torch.float32, torch.float32),
                                              (50, 20, torch.bfloat16, torch.bfloat16), (7, 0, torch.float32, torch.float32)])
def test_gradients_of_the_norms_stay_inside(D, R, dtype, gdtype):
    """Guard bands around the gradients and the workspace, through the C entry point."""
    import ctypes

    import kimi_delta_attention_21_b200 as K
    from kimi_delta_attention_21_b200 import _lib as L
    lib, code = K.load_library(), lambda t: L.KDA_F32 if t == torch.float32 else L.KDA_BF16
    B, S, Hq, Hk = 2, 301, 3, 2
    g = gen(D)
    q, k = randn(g, B, S, Hq, D, dtype=dtype), randn(g, B, S, Hk, D, dtype=dtype)
    dyq, dyk = randn(g, B, S, Hq, D, dtype=gdtype), randn(g, B, S, Hk, D, dtype=gdtype)
    qw, kw = 1 + randn(g, D), 1 + randn(g, D)
    pos, inv = torch.arange(B * S, device="cuda").view(B, S), torch.logspace(0, -3, max(R // 2, 1), device="cuda")
    f = L.QkNormArgs(B=B, S=S, H_q=Hq, H_k=Hk, D=D, dtype=code(dtype), q=q.data_ptr(), k=k.data_ptr(), q_stride_b=S * Hq * D,
                     q_stride_s=Hq * D, k_stride_b=S * Hk * D, k_stride_s=Hk * D, norm=L.NORM_RMS, eps=1e-6,
                     q_weight=qw.data_ptr(), k_weight=kw.data_ptr(), positions=pos.data_ptr(), inv_freq=inv.data_ptr(), rot_dim=R,
                     stream=torch.cuda.current_stream().cuda_stream)
    a = L.QkNormBwdArgs(fwd=f, grad_dtype=code(gdtype), dq_out=dyq.data_ptr(), dk_out=dyk.data_ptr())
    bufs = dict(dq=Guarded(q.shape, dtype), dk=Guarded(k.shape, dtype), dq_weight=Guarded((D,), torch.float32),
                dk_weight=Guarded((D,), torch.float32))
    for n, b in bufs.items():
        setattr(a, n, b.t.data_ptr())
    n = ctypes.c_size_t(0)
    assert lib.kda_qk_norm_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    bufs["workspace"] = Guarded((n.value // 4,), torch.float32)
    a.workspace, a.workspace_bytes = bufs["workspace"].t.data_ptr(), n.value
    assert lib.kda_qk_norm_bwd(ctypes.byref(a)) == 0, lib.kda_last_error()
    for what, b in bufs.items():
        b.check(what)
    want = K.qk_norm_bwd(q, k, dyq, dyk, norm="rms", q_weight=qw, k_weight=kw, **(dict(positions=pos, inv_freq=inv) if R else {}))
    for what, t in want.items():
        assert torch.equal(bufs[what].t, t), what

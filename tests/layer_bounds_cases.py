"""Every way through the operators around the gated delta rule, one call each with its outputs, for the test of the checked
build and its child process.  As a script: `python tests/layer_bounds_cases.py OUT.npz [last]` runs them on the library that
KDA_LIBRARY picks and saves every output, or, with `last`, how many writes each call skipped and whether the last element of
each of its outputs was left as it was."""
import ctypes
import os
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
for p in (os.path.dirname(HERE), HERE):
    if p not in sys.path:
        sys.path.insert(0, p)


def calls():
    """(name, call) pairs; a call gives its outputs by name.  Buffers that the call is handed are filled with NaN first."""
    import torch

    import kimi_delta_attention_21_b200 as K
    from layer_testlib import gen, randn, unit
    bf, f32, nan = torch.bfloat16, torch.float32, float("nan")
    pos = lambda B, S: torch.arange(B * S, device="cuda").view(B, S)
    freq = lambda R: torch.logspace(0, -3, R // 2, device="cuda")
    full = lambda shape, dt: torch.full(shape, nan, device="cuda", dtype=dt)
    out = []

    # norms: whole vectors, and any size; enough rows that every CTA of the backward has some
    for D, R, H, dt in ((128, 128, 3, bf), (64, 0, 2, f32), (256, 128, 1, f32), (50, 20, 2, bf), (33, 0, 1, f32)):
        def qk(D=D, R=R, H=H, dt=dt, bwd=False):
            g, (B, S) = gen(D), (2, 4000)
            q, k = randn(g, B, S, H, D, dtype=dt), randn(g, B, S, H, D, dtype=dt)
            kw = dict(norm="rms", q_weight=1 + randn(g, D), k_weight=1 + randn(g, D))
            if R:
                kw.update(positions=pos(B, S), inv_freq=freq(R))
            if not bwd:
                o = [full(q.shape, dt), full(k.shape, dt)]
                K.qk_norm(q, k, out_q=o[0], out_k=o[1], **kw)
                return dict(zip(("q", "k"), o))
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            ws = full((2 * sms * 2 * D,), f32)  # two CTAs an SM and side, a row of D sums each
            r = K.qk_norm_bwd(q, k, randn(g, B, S, H, D), randn(g, B, S, H, D), workspace=ws.view(torch.uint8), **kw)
            return dict(r, workspace=ws)
        out += [(f"qk_norm{D}", qk), (f"qk_norm_bwd{D}", lambda qk=qk: qk(bwd=True))]

    # decode: whole vectors and not, each number of rows a warp; pools and their first states
    for Dk, Dv, T, dt in ((128, 128, 1, bf), (128, 128, 3, f32), (96, 72, 2, bf), (60, 50, 1, f32), (20, 13, 4, bf), (16, 16, 1, bf)):
        def dec(Dk=Dk, Dv=Dv, T=T, dt=dt):
            g, B, H = gen(Dk + T), 3, 2
            state, o = randn(g, B, H, Dk, Dv), full((B, T, H, Dv), dt)
            if last:
                state = full(state.shape, f32)
            K.gdn_decode_step(unit(g, B, T, H, Dk, dtype=dt), unit(g, B, T, H, Dk, dtype=dt), randn(g, B, T, H, Dv, dtype=dt),
                              torch.rand((B, T, H), generator=g, device="cuda").to(dt), state,
                              z=randn(g, B, T, H, dtype=dt), out=o)
            return dict(o=o, **({} if last else {"state": state}))
        out.append((f"decode{Dk}_{Dv}_{T}", dec))

    # gradients of the gated delta rule: pairs of columns and odd ones
    for S, Dk, Dv, dt in ((200, 128, 128, bf), (130, 40, 72, f32), (70, 33, 51, bf), (64, 17, 9, f32)):
        def bwd(S=S, Dk=Dk, Dv=Dv, dt=dt):
            g, B, H = gen(S), 2, 2
            s0 = randn(g, B, H, Dk, Dv)
            return K.gdn_chunk_bwd(unit(g, B, S, H, Dk, dtype=dt), unit(g, B, S, H, Dk, dtype=dt), randn(g, B, S, H, Dv, dtype=dt),
                                   torch.rand((B, S, H), generator=g, device="cuda").to(dt), randn(g, B, S, H, Dv, dtype=dt),
                                   z=randn(g, B, S, H, dtype=dt), initial_state=s0, d_final_state=s0)
        out.append((f"gdn_bwd{S}", bwd))

    # quantisers: rows of whole blocks, of whole vectors, of any size; blocks of 128 rows alike
    for N, Kd, rows, dt in ((40, 256, 1, bf), (40, 264, 1, f32), (40, 130, 1, bf), (200, 256, 128, f32), (200, 130, 128, bf)):
        def quant(N=N, Kd=Kd, rows=rows, dt=dt):
            return dict(zip(("x8", "scale"), K.quant_fp8(randn(gen(Kd), N, Kd, dtype=dt), rows)))
        out.append((f"quant{Kd}_{rows}", quant))
    for N, H, Dv, dt in ((40, 2, 128, bf), (40, 3, 64, f32), (40, 3, 48, bf), (40, 40, 48, bf), (20, 100, 48, bf), (40, 3, 50, f32)):
        def ng(N=N, H=H, Dv=Dv, dt=dt):
            g = gen(H)
            return dict(zip(("x8", "scale"), K.norm_gate_fp8(randn(g, N, H, Dv, dtype=dt), randn(g, N, H, Dv, dtype=dt))))
        out.append((f"norm_gate{H}_{Dv}", ng))

    # projection: few rows (whole vectors and not), many rows without a map for the stores, any K
    for N, Kd, M, dt in ((70, 256, 264, bf), (70, 256, 67, f32), (2600, 256, 2047, bf), (70, 130, 67, f32)):
        def proj(N=N, Kd=Kd, M=M, dt=dt):
            g = gen(N + M)
            x, w = K.quant_fp8(randn(g, N, Kd)), K.quant_fp8(randn(g, M, Kd), 128)
            reset()
            y = full((N, M), dt)
            K.out_proj_fp8(*x, *w, out_dtype=dt, out=y)
            return dict(y=y)
        out.append((f"proj{N}_{Kd}_{M}", proj))
    return out


last = False


def counter(reset=0):
    import torch

    import kimi_delta_attention_21_b200 as K
    torch.cuda.synchronize()
    n, chk = ctypes.c_uint32(0), ctypes.c_int(-1)
    assert K.load_library().kda_device_bounds_errors(ctypes.byref(n), reset, ctypes.cast(ctypes.pointer(chk), ctypes.c_void_p)) == 0
    return n.value, chk.value


def reset():
    counter(1)


def run_cases():
    """Every output of every call, and the counter."""
    res = {}
    reset()
    for name, call in calls():
        res.update({f"{name}/{n}": t.float().cpu().numpy() for n, t in call().items()})
    return res, counter(1)


def run_last():
    """name -> (writes skipped, names of the outputs whose last element was written all the same)"""
    import torch
    global last
    last = True
    # what the calls allocate is NaN until it is written
    torch.use_deterministic_algorithms(True, warn_only=True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    res = {}
    for name, call in calls():
        reset()
        outs = call()
        n = counter(1)[0]
        res[name] = (n, ",".join(o for o, t in outs.items() if not bool(t.flatten()[-1].float().isnan())))
    return res


if __name__ == "__main__":
    if sys.argv[2:] == ["last"]:
        np.savez(sys.argv[1], **{n: np.array([str(c), o]) for n, (c, o) in run_last().items()})
    else:
        arrays, (errors, checked) = run_cases()
        np.savez(sys.argv[1], **arrays, _errors=np.array(errors), _checked=np.array(checked))

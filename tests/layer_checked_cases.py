"""The operators around the gated delta rule on seeded inputs, for the checked-build test and the child process that
runs them on libkda_checked.so.  As a script: `python tests/layer_checked_cases.py OUT.npz` (KDA_LIBRARY picks the
library)."""
import ctypes
import os
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
for p in (os.path.dirname(HERE), HERE):
    if p not in sys.path:
        sys.path.insert(0, p)


def run_cases():
    import torch

    import kimi_delta_attention_21_b200 as K
    from layer_testlib import gen, randn, unit
    out = {}

    def keep(name, t):
        out[name] = t.detach().float().cpu().numpy()

    for dtype, Dk, Dv, S in ((torch.bfloat16, 128, 128, 200), (torch.float32, 40, 72, 130)):
        g = gen(S)
        B, H = 2, 3
        q, k = unit(g, B, S, H, Dk, dtype=dtype), unit(g, B, S, H, Dk, dtype=dtype)
        v, do = randn(g, B, S, H, Dv, dtype=dtype), randn(g, B, S, H, Dv, dtype=dtype)
        beta, z = torch.rand((B, S, H), generator=g, device="cuda").to(dtype), randn(g, B, S, H, dtype=dtype)
        s0 = randn(g, B, H, Dk, Dv)
        r = K.gdn_chunk_bwd(q, k, v, beta, do, z=z, initial_state=s0, d_final_state=s0 * 0.5)
        for n, t in r.items():
            keep(f"bwd{S}_{n}", t)
        pool = randn(g, 5, H, Dk, Dv)
        slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
        at = lambda t: t[:, :4].contiguous()
        keep(f"dec{S}_o", K.gdn_decode_step(at(q), at(k), at(v), at(beta), pool, z=at(z), gate_logits=at(do), slots=slots))
        keep(f"dec{S}_state", pool)
        x8, sc = K.norm_gate_fp8(v, do)
        keep(f"ng{S}_x", x8)
        keep(f"ng{S}_s", sc)
        W8, Ws = K.quant_fp8(randn(g, 80, H * Dv, std=0.1), 128)
        keep(f"proj{S}", K.out_proj_fp8(x8, sc, W8, Ws))
        qn, kn = K.qk_norm(v, do)
        keep(f"qn{S}", qn)
        keep(f"kn{S}", kn)
    torch.cuda.synchronize()
    lib, n, chk = K.load_library(), ctypes.c_uint32(0), ctypes.c_int(-1)
    assert lib.kda_device_bounds_errors(ctypes.byref(n), 1, ctypes.cast(ctypes.pointer(chk), ctypes.c_void_p)) == 0
    return out, {"bounds_errors": n.value, "checked_build": chk.value}


if __name__ == "__main__":
    arrays, counters = run_cases()
    np.savez(sys.argv[1], **arrays, **{"_" + n: np.array(v) for n, v in counters.items()})

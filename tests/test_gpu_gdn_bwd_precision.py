"""The gradients of the gated delta rule against 64 bits in the norm, where the bound is a few times what they reach (element by
element, test_gpu_gdn_bwd.py)."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_gdn_bwd import BF16, F32, gradients64, make  # noqa: E402

pytestmark = pytest.mark.gpu

# A split operand's lo part is at most 2^-12 of it and is cut to 11 bits by the product: a term of a product is off by 2^-23 of
# itself in each operand; the tensor core cuts 16 partial sums of 24 bits: as random steps 2^-22 together.  Eight products in a
# row, independent: sqrt(8) 2^-21.5 = 2^-20 of the norm.  Four times that, for the norm of (I + A)^-1 and its transpose, which
# the errors of U, W, dBv and dBk pass through.
REL = 2.0 ** -18


@pytest.mark.parametrize("B,S,H,Dk,Dv,dtype,decay,g_min", [
    (2, 130, 3, 128, 128, BF16, "z", -5.0), (1, 200, 2, 128, 128, F32, "log", -0.25), (2, 300, 2, 72, 100, F32, "log", -1.0),
    (1, 320, 2, 128, 128, BF16, "z", -0.25), (3, 63, 2, 64, 32, BF16, "log", -1.0), (2, 129, 2, 33, 17, F32, "z", -20.0)])
def test_norm_of_the_error(B, S, H, Dk, Dv, dtype, decay, g_min):
    import kimi_delta_attention_21_b200 as K
    d, opt = make(B, S, H, Dk, Dv, dtype, decay, g_min, True, seed=S)
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=g_min, **opt)
    for n, want in gradients64(d, opt, g_min).items():
        err = float((got[n].double() - want).norm() / want.norm())
        assert err <= REL, f"{n}: {err:.2e}"

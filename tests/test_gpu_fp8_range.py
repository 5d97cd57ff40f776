"""The fused norm, gate and quantisation of fp32 heads whose squares fp32 does not hold, large and small: as the unquantised
norm and gate, whose sums are fp64 too."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import assert_within, gen, randn  # noqa: E402
from test_gpu_fp8_precision import definition, scales_of, slack  # noqa: E402

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-18, 1e18, 1e25, 1e37])
@pytest.mark.parametrize("H,Dv", [(2, 128), (3, 64), (7, 48), (3, 50)])
def test_heads_of_any_size(H, Dv, size):
    import kimi_delta_attention_21_b200 as K
    g = gen(H)
    o, gate = randn(g, 9, H, Dv) * size, randn(g, 9, H, Dv)
    _, sc = K.norm_gate_fp8(o, gate, eps=0.0)
    want, t = scales_of(definition(o, gate, 0.0)), slack(Dv, F32)
    assert_within(sc, want, t * want, "scale")
    y = K.norm_gate(o, gate, eps=0.0).flatten(1)
    # the unquantised values are within as much of the definition (their own roundings: no more than the ones counted there)
    assert_within(scales_of(y.double()), want, t * want, "norm and gate")

"""The fused norm, gate and quantisation forms its values as the definition says: the precise sigmoid (gates far from zero,
infinite and NaN ones), the quotient by the scale, fp64 sums of fp32 inputs; counted in half-steps of fp32, not of e4m3."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import U32, assert_within, gen, randn  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

# each way through the entry point: whole blocks, power-of-two heads with a ragged edge, heads that straddle the blocks
# (whole vectors, by 64 to 256 threads a token), and any others
SHAPES = [(40, 4, 128), (33, 3, 64), (50, 7, 48), (20, 16, 80), (6, 200, 48), (30, 9, 50), (5, 2, 300)]


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def definition(o, gate, eps):
    o = o.double()
    return (o / (o.square().mean(-1, keepdim=True) + eps).sqrt() * torch.sigmoid(gate.double())).flatten(1)


def scales_of(x):
    N, W = x.shape
    p = torch.nn.functional.pad(x, (0, -W % 128)).view(N, -1, 128)
    amax = p.abs().nan_to_num(0.0).amax(-1)
    return torch.where(amax > 0, (amax / 448).clamp_min(2.0 ** -126), torch.ones_like(amax))


def slack(Dv, dtype):
    """Half-steps of fp32 that a value x can be off by, relative to it.  Fixed: the sigmoid 8 (its exponential 2 units = 4,
    1 + e one, the reciprocal one unit = 2, e times it one), its product with o and 1 / rms two, the root's reciprocal 2 units = 4, mean
    and eps 3, the division by 448 one: 18.  The sum of squares (bf16: each square is exact, the sum fp32) as many as it has
    additions in a row, halved by the root; 8 a vector, then at most D_v / 8 in a row."""
    return (18 + (0 if dtype == F32 else (8 + Dv / 8) / 2)) * U32


def nearest(q):
    return q.float().to(E4M3).double()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,Dv", SHAPES)
@pytest.mark.parametrize("mean", [0.0, -20.0, -60.0, -80.0])
def test_values_and_scales_to_fp32_accuracy(K, N, H, Dv, dtype, mean):
    g = gen(N + H + Dv)
    o, gate = randn(g, N, H, Dv, dtype=dtype, std=0.3), (randn(g, N, H, Dv) + mean).to(dtype)
    x8, sc = K.norm_gate_fp8(o, gate, eps=1e-5)
    x, t = definition(o, gate, 1e-5), slack(Dv, dtype)
    want = scales_of(x)
    assert_within(sc, want, t * want, "scale")
    # the quotient: x, the scale and the division (one half-step) each off by as much at most; the value has to be the
    # nearest to some number within that of x / scale
    q = x / want.repeat_interleave(128, 1)[:, :x.shape[1]]
    lo, hi, v = nearest(q * (1 - 2 * t - 2 * U32)), nearest(q * (1 + 2 * t + 2 * U32)), x8.float().double()
    bad = (v != lo) & (v != hi)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} values are not the nearest"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Dv", [128, 48, 50])
def test_gates_at_the_ends(K, Dv, dtype):
    """Infinite, NaN and far gates: sigmoid(-88) = 6e-39 is half the smallest scale, sigmoid(-100) = 4e-44 far below it."""
    inf = float("inf")
    rows = [[inf] * Dv, [-inf] * Dv, [100.0] * Dv, [-100.0] * Dv, [-88.0] * Dv, [88.0] * Dv, [float("nan")] * Dv,
            [0.0, -inf, inf, float("nan"), 88.0, -100.0] + [1.0] * (Dv - 6)]
    gate = torch.tensor(rows, device="cuda")[:, None].to(dtype)
    o = (randn(gen(Dv), len(rows), 1, Dv).abs() + 0.5).to(dtype)
    x8, sc = K.norm_gate_fp8(o, gate)
    v, x = x8.float().double(), definition(o, gate, 1e-6)
    assert torch.equal(v.isnan(), x.isnan())
    assert bool((sc[1] == 1).all()) and bool((sc[6] == 1).all()) and bool((v[1] == 0).all()) and bool((v[3] == 0).all())
    assert bool((sc[3:5] == 2.0 ** -126).all()) and bool((v[4] > 0).any())
    want, t = scales_of(x), slack(Dv, dtype)
    assert_within(sc, want, t * want, "scale")
    # below 2^-126 fp32's steps are 2^-149 each: two of them (sigmoid, product) beside the relative error
    q = x / want
    e = q.abs() * (2 * t + 2 * U32) + 2 * 2.0 ** -149 / want
    lo, hi = nearest(q - e), nearest(q + e)
    assert bool(((v == lo) | (v == hi) | x.isnan()).all())


def test_many_fp32_heads(K):
    """As many heads as the entry point takes, of no whole vector."""
    o, gate = randn(gen(1), 2, 8192, 3), randn(gen(2), 2, 8192, 3)
    x8, sc = K.norm_gate_fp8(o, gate)
    want, t = scales_of(definition(o, gate, 1e-6)), slack(3, F32)
    assert_within(sc, want, t * want, "scale")

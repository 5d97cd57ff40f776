"""Infinite and NaN elements of channels that the rotation leaves alone stay in their channel, where the definition keeps
them: in the forward (an infinite element makes the row's scale zero, and itself NaN) and in the sums that are the weights'
gradients."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import U32, assert_within, gen, half_step, randn  # noqa: E402
from test_gpu_qk_norm import forward64, tolerance, turn  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


# whole vectors (one or two a lane) and the kernel for any size; R ends on a vector, inside one, inside a pair's reach
CASES = [(128, 64, False, BF16), (128, 64, True, BF16), (128, 68, True, BF16), (256, 128, False, F32), (256, 130, True, F32),
         (64, 32, True, F32), (96, 32, False, BF16), (50, 20, True, BF16), (50, 20, False, F32)]


def inputs(D, R, dtype, seed):
    g = gen(seed)
    x = randn(g, 1, 12, 2, D, dtype=dtype)
    pos = torch.randint(0, 5000, (1, 12), generator=g, device="cuda")
    inv = (10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)).float()
    return g, x, 1 + randn(g, D, std=0.2), pos, inv


@pytest.mark.parametrize("norm", ["l2", "rms"])
@pytest.mark.parametrize("D,R,inter,dtype", CASES)
def test_forward(K, D, R, inter, dtype, norm):
    g, x, w, pos, inv = inputs(D, R, dtype, D + R)
    for row, c in ((1, R), (2, R + 1), (3, D - 1), (4, D - 2)):  # either side of a pair's place
        x[0, row, 0, c] = INF if row % 2 else -INF
    x[0, 5, 1, R] = NAN
    y, _ = K.qk_norm(x, x, norm=norm, q_weight=w, positions=pos, inv_freq=inv, interleaved=inter)
    want = forward64(x, w, norm, 1e-6, R, inter, pos, inv)
    assert int(want.isnan().sum()) == 4 + D  # one element of each infinite row, the row with the NaN
    assert_within(y, want, tolerance(want.nan_to_num(0.0), dtype), "y")


@pytest.mark.parametrize("D,R,inter,dtype", CASES)
def test_weight_gradients(K, D, R, inter, dtype):
    g, x, w, pos, inv = inputs(D, R, dtype, D + R + 1)
    for bad in (INF, NAN):
        for c in (R, R + 1, D - 1):
            dy = randn(g, *x.shape)
            dy[0, 3, 1, c] = bad
            got = K.qk_norm_bwd(x, x, dy, dy, norm="rms", q_weight=w, k_weight=w, positions=pos, inv_freq=inv, interleaved=inter)
            x64 = x.double()
            y = x64 / (x64.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            dw = (turn(dy.double(), R, inter, pos, inv, sign=-1.0) * y).sum((0, 1, 2))
            ok = torch.arange(D, device="cuda") != c
            for n in ("dq_weight", "dk_weight"):
                # a sum over 24 rows, each term off by half-steps of 2 max |dy| |y| (the turn mixes two channels)
                size = (2 * dy.double().nan_to_num(0.0, 0.0, 0.0).abs().amax(-1, keepdim=True) * y.abs()).sum((0, 1, 2))
                assert_within(got[n][ok], dw[ok], ((24 + 64) * U32 * size)[ok], n)
                assert torch.equal(got[n][c].isnan(), dw[c].isnan()) and (bad != INF or float(got[n][c]) == float(dw[c])), n

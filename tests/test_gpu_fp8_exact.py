"""The e4m3 projection accumulates in 24 bits: products and sums that are whole numbers below 2^24 come out exactly, on the
tensor cores and on the SIMT kernel.  An accumulator of fewer bits, or products cut as they are aligned, would lose the ones
beside the large terms."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import gen  # noqa: E402

pytestmark = pytest.mark.gpu
F32, E4M3 = torch.float32, torch.float8_e4m3fn
SHAPES = [(5, 128, 64), (64, 4096, 256), (300, 1040, 129), (2600, 512, 2049), (3000, 4096, 2048), (70, 130, 67)]


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def whole(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").float()


def product(K, x, w, xs, ws):
    x8, w8 = x.to(E4M3), w.to(E4M3)
    assert torch.equal(x8.float(), x) and torch.equal(w8.float(), w)
    return K.out_proj_fp8(x8, xs, w8, ws, out_dtype=F32).double()


@pytest.mark.parametrize("N,Kd,M", SHAPES)
def test_sums_of_whole_numbers(K, N, Kd, M):
    """Both signs up to 15, all blocks: |sum| <= 4096 * 225 < 2^20; scales are powers of two that keep it below 2^24."""
    g, kb = gen(N + Kd), -(-Kd // 128)
    x, w = whole(g, -15, 15, N, Kd), whole(g, -15, 15, M, Kd)
    xs, ws = 2.0 ** whole(g, 0, 2, N, kb), 2.0 ** whole(g, 0, 2, -(-M // 128), kb)
    a = x.double() * xs.double().repeat_interleave(128, 1)[:, :Kd]
    b = w.double() * ws.double().repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :Kd]
    assert torch.equal(product(K, x, w, xs, ws), a @ b.mT)


@pytest.mark.parametrize("big", [240.0, 448.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("N,M", [(5, 64), (300, 129), (2600, 2049)])
def test_ones_beside_the_largest_products(K, N, M, sign, big):
    """One block: up to 72 products of the largest values (448^2 = 200704; 72 of them below 2^24) beside products of 0 to 3,
    which a sum of 22 bits would lose; with both signs they cancel but for those."""
    g, Kd = gen(N + M), 128
    large = torch.rand((1, Kd), generator=g, device="cuda").argsort(1) < 72
    turn = torch.where(torch.arange(Kd, device="cuda") % 2 == 0, 1.0, sign)
    x, w = torch.where(large, turn * big, whole(g, 0, 1, N, Kd)), torch.where(large, torch.tensor(big, device="cuda"), whole(g, 1, 3, M, Kd))
    want = x.double() @ w.double().mT
    assert float((x.double().abs() @ w.double().abs().mT).max()) < 2 ** 24
    ones = torch.ones(1, 1, device="cuda")
    assert torch.equal(product(K, x, w, ones.expand(N, 1).contiguous(), ones.expand(-(-M // 128), 1).contiguous()), want)

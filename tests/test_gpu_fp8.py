"""The e4m3 output path: quantisers against the definition (values, scales,
edge blocks, zeros, non-finite elements) and the product of quantised operands
against 64 bits over odd sizes, both engines, and the three in a row against the
bf16 path."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import U32, Guarded, assert_within, captured, gen, half_step, randn  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
STEP8 = 2.0 ** -4  # half a step of e4m3, relative to the value


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def blocks(x, rows):
    """(N, K) as (n, rows, kb, 128) with zeros behind the edges."""
    N, Kd = x.shape
    p = torch.zeros(-(-N // rows) * rows, -(-Kd // 128) * 128, dtype=x.dtype, device=x.device)
    p[:N, :Kd] = x
    return p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128)


def spread(scale, rows, N, Kd):
    return scale.repeat_interleave(rows, 0)[:N].repeat_interleave(128, 1)[:, :Kd]


def check_quantised(x, x8, scales, rows, slack):
    """Every scale is its block's largest magnitude over 448, every value the e4m3 nearest to x / scale: off by at most
    half a step (2^-4 of the value; below e4m3's normal range, half of 2^-9)."""
    x = x.double()
    amax = blocks(x, rows).abs().amax((1, 3))
    want = torch.where(amax > 0, (amax / 448).clamp_min(2.0 ** -126), torch.ones_like(amax))
    assert_within(scales, want, (4 * U32 + slack) * want, "scale")
    s = spread(scales.double(), rows, *x.shape)
    near = torch.maximum(STEP8 * (x / s).abs(), torch.tensor(2.0 ** -10, device=x.device, dtype=torch.float64))
    assert_within(x8.float(), x / s, near * (1 + 2 ** -10) + slack * (x / s).abs(), "value")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Kd,rows", [(1, 1, 1), (3, 128, 1), (37, 1000, 1), (300, 4096, 1), (128, 128, 128), (1, 5, 128),
                                       (300, 1000, 128), (257, 513, 128)])
def test_quantises(K, N, Kd, rows, dtype):
    g = gen(N + Kd)
    x = randn(g, N, Kd, dtype=dtype) * torch.logspace(-6, 3, N, device="cuda", dtype=F32)[:, None].to(dtype)
    x8, sc = K.quant_fp8(x, rows)
    assert x8.dtype == E4M3 and x8.shape == x.shape
    check_quantised(x, x8, sc, rows, 0.0)
    s = spread(sc, rows, N, Kd)  # the division is IEEE's: the value is exactly the nearest
    assert torch.equal(x8.float(), (x.float() / s).to(E4M3).float())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,Kd,off", [(37, 1001, 0), (9, 130, 0), (64, 256, 1), (5000, 264, 0)])
def test_quantises_rows_of_any_alignment(K, N, Kd, off, dtype):
    x = randn(gen(Kd), N * Kd + off, dtype=dtype)[off:].view(N, Kd)
    x8, sc = K.quant_fp8(x)
    check_quantised(x, x8, sc, 1, 0.0)
    assert torch.equal(x8.float(), (x.float() / spread(sc, 1, N, Kd)).to(E4M3).float())


def test_blocks_of_zeros_and_non_finite(K):
    x = torch.zeros(4, 300, device="cuda")
    x[1, 5], x[1, 6] = float("nan"), 2.0
    x[2, 200], x[2, 201] = float("inf"), 3.0
    x[3, 10] = 1e-40                              # its scale would be below fp32's normal range
    x8, sc = K.quant_fp8(x)
    assert bool((sc[0] == 1).all()) and bool((x8[0].float() == 0).all())
    assert bool(x8[1, 5].float().isnan()) and float(x8[1, 6].float()) == 448 and float(sc[1, 0]) == pytest.approx(2 / 448)
    assert bool(sc[2, 1].isinf()) and bool(x8[2, 200].float().isnan()) and float(x8[2, 201].float()) == 0
    assert float(sc[3, 0]) == 2.0 ** -126 and bool(x8[3].float().isfinite().all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,Dv", [(1, 1, 128), (7, 5, 128), (256, 32, 128), (33, 3, 64), (5, 7, 48), (9, 3, 100), (2, 2, 300),
                                    (4, 1, 1), (3, 131, 16), (6, 48, 96), (3, 200, 48), (2, 85, 104)])
def test_norm_gate_quantises_its_result(K, N, H, Dv, dtype):
    g = gen(N * H + Dv)
    o, gate = randn(g, N, H, Dv, dtype=dtype, std=0.3), randn(g, N, H, Dv, dtype=dtype, std=2.0)
    x8, sc = K.norm_gate_fp8(o, gate, eps=1e-5)
    o64 = o.double()
    x = (o64 / (o64.square().mean(-1, keepdim=True) + 1e-5).sqrt() * torch.sigmoid(gate.double())).flatten(1)
    # the norm (a sum of D_v squares, a root), the sigmoid and three products in fp32: under 64 half-steps
    check_quantised(x, x8, sc, 1, 64 * U32)


def test_norm_gate_writes_stay_inside(K):
    """Guard bands, through the C entry point (its outputs are the caller's buffers)."""
    lib = K.load_library()
    for N, H, Dv in ((5, 3, 128), (4, 3, 40)):
        o, gate = randn(gen(1), N, H, Dv, dtype=BF16), randn(gen(2), N, H, Dv, dtype=BF16)
        g8, gs = Guarded((N, H * Dv), torch.uint8), Guarded((N, -(-H * Dv // 128)), F32)
        st = torch.cuda.current_stream().cuda_stream
        assert lib.kda_norm_gate_fp8(o.data_ptr(), gate.data_ptr(), N, H, Dv, 1e-6, 1, g8.t.data_ptr(), gs.t.data_ptr(),
                                     st) == 0
        g8.check("x8")
        gs.check("scales")
        x8, sc = K.norm_gate_fp8(o, gate)
        assert torch.equal(g8.t, x8.view(torch.uint8)) and torch.equal(gs.t, sc)


def test_quantiser_and_projection_writes_stay_inside(K):
    lib, st = K.load_library(), torch.cuda.current_stream().cuda_stream
    for N, Kd, rows in ((5, 264, 1), (7, 130, 1), (131, 264, 128), (131, 130, 128)):
        x = randn(gen(Kd), N, Kd, dtype=BF16)
        g8, gs = Guarded((N, Kd), torch.uint8), Guarded((-(-N // rows), -(-Kd // 128)), F32)
        assert lib.kda_quant_fp8(x.data_ptr(), 1, N, Kd, rows, g8.t.data_ptr(), gs.t.data_ptr(), st) == 0
        g8.check("x8")
        gs.check("scales")
    for N, Kd, M in ((5, 256, 67), (300, 512, 2000), (2600, 256, 2048), (9, 130, 70)):
        x, xs, w, ws = operands(N, Kd, M)
        y = Guarded((N, M), BF16)
        assert lib.kda_out_proj_fp8(x.data_ptr(), xs.data_ptr(), w.data_ptr(), ws.data_ptr(), N, Kd, M, y.t.data_ptr(), 1,
                                    st) == 0
        y.check("y")
        assert torch.equal(y.t, K.out_proj_fp8(x, xs, w, ws))


@pytest.mark.parametrize("rows", [1, 128])
def test_quotients_at_extreme_scales(K, rows):
    """Scales from the smallest normal value to the largest: the value is the nearest to IEEE's quotient at all of them."""
    e = torch.arange(-140, 127, device="cuda", dtype=F32)
    top = torch.exp2(e).repeat_interleave(rows)
    x = torch.rand((top.numel(), 128), generator=gen(7), device="cuda") * 2 - 1
    x[::rows, 0] = 1.0
    x = x * top[:, None]
    x8, sc = K.quant_fp8(x, rows)
    s = spread(sc, rows, *x.shape)
    assert torch.equal(x8.float(), (x / s).to(E4M3).float())


def operands(N, Kd, M, seed=0):
    """e4m3 operands whose scales differ from block to block by powers of ten."""
    g = gen(seed)
    x = torch.randn((N, Kd), generator=g, device="cuda").clamp(-4, 4).mul(60).to(E4M3)
    w = torch.randn((M, Kd), generator=g, device="cuda").clamp(-4, 4).mul(60).to(E4M3)
    kb = -(-Kd // 128)
    xs = 10.0 ** (torch.rand((N, kb), generator=g, device="cuda") * 3 - 3)
    ws = 10.0 ** (torch.rand((-(-M // 128), kb), generator=g, device="cuda") * 3 - 3)
    return x, xs, w, ws


def product64(x, xs, w, ws):
    (N, Kd), M = x.shape, w.shape[0]
    a = x.double() * spread(xs.double(), 1, N, Kd)
    b = w.double() * spread(ws.double(), 128, M, Kd)
    return a @ b.mT, a.abs() @ b.abs().mT


# a block of 128 products accumulated in fp32 (e4m3 products have 8 bits: exact), then K / 128 scaled additions: each
# sum is off by at most its number of additions times half a step of fp32, relative to the sum of magnitudes; the tensor
# core's accumulator may drop bits below 2^-22 of the block's largest partial sum, 128 times: 2^-15 of the magnitudes
def tolerance(want, size, Kd, dtype):
    return half_step(dtype) * want.abs() * (1 + 2 ** -7) + (2 ** -15 + (Kd / 128 + 8) * U32) * size


SIZES = [(1, 128, 64), (1, 16, 8), (5, 128, 256), (64, 4096, 4096), (130, 272, 136), (200, 1040, 1000), (257, 384, 520),
         (300, 2048, 2048), (33, 4096, 264), (1000, 640, 4096), (2500, 512, 4104), (128, 8192, 128), (20, 4240, 512),
         (1, 2048, 4096), (20, 1168, 520), (1500, 1040, 2000)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,Kd,M", SIZES)
def test_product_on_the_tensor_cores(K, N, Kd, M, out):
    x, xs, w, ws = operands(N, Kd, M, seed=N + M)
    gy = Guarded((N, M), out)
    K.out_proj_fp8(x, xs, w, ws, out_dtype=out, out=gy.t)
    gy.check("y")
    want, size = product64(x, xs, w, ws)
    assert_within(gy.t, want, tolerance(want, size, Kd, out), "y")
    import ctypes
    n = ctypes.c_uint32(0)
    assert K.load_library().kda_device_timeouts(ctypes.byref(n), 1) == 0 and n.value == 0


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,Kd,M", [(1, 1, 1), (3, 130, 5), (65, 200, 67), (70, 136, 129), (30, 1000, 300)])  # K % 16
def test_product_on_the_simt_kernel(K, N, Kd, M, out):
    x, xs, w, ws = operands(N, Kd, M, seed=N + M)
    gy = Guarded((N, M), out, offset=1)
    K.out_proj_fp8(x, xs, w, ws, out_dtype=out, out=gy.t)
    gy.check("y")
    want, size = product64(x, xs, w, ws)
    assert_within(gy.t, want, tolerance(want, size, Kd, out), "y")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,Kd,M", [(1, 128, 1), (5, 272, 67), (300, 1040, 129), (2600, 512, 2049), (2600, 256, 2047)])
def test_product_with_rows_off_sixteen_bytes(K, N, Kd, M, out):
    x, xs, w, ws = operands(N, Kd, M, seed=N + M)
    for offset in (0, 1):
        gy = Guarded((N, M), out, offset=offset)
        K.out_proj_fp8(x, xs, w, ws, out_dtype=out, out=gy.t)
        gy.check("y")
        want, size = product64(x, xs, w, ws)
        assert_within(gy.t, want, tolerance(want, size, Kd, out), "y")


def test_non_finite_rows_stay_in_their_row_and_column(K):
    x, xs, w, ws = operands(140, 256, 264, seed=3)
    xs[7, 1] = float("nan")
    ws[1, 0] = float("inf")
    x8 = x.view(torch.uint8)
    x8[9, 100] = 0x7F                                # e4m3's NaN
    y = K.out_proj_fp8(x, xs, w, ws, out_dtype=F32)
    ok = torch.ones(140, dtype=torch.bool, device="cuda")
    ok[[7, 9]] = False
    assert bool(y[ok][:, :128].isfinite().all()) and bool(y[ok][:, 256:].isfinite().all())
    assert not bool(y[:, 128:256].isfinite().any())
    assert bool(y[7].isnan().all()) and bool(y[9].isnan().all())


def test_whole_path_against_the_bf16_one(K):
    """norm + gate + quantisation + product, against the same layer output in bf16: the quantisation's own error is a
    random half-step of e4m3 in each factor, 2^-4 / sqrt(3) each, averaged over K terms."""
    g = gen(11)
    N, H, Dv, Dm = 300, 16, 128, 2048
    o, gate = randn(g, N, H, Dv, dtype=BF16, std=0.2), randn(g, N, H, Dv, dtype=BF16)
    W = randn(g, Dm, H * Dv, dtype=BF16, std=(H * Dv) ** -0.5)
    W8, Ws = K.quant_fp8(W, 128)
    x8, xs = K.norm_gate_fp8(o, gate)
    y = K.out_proj_fp8(x8, xs, W8, Ws)
    ref = K.out_norm_gate_proj(o, gate, W)
    assert y.shape == (N, Dm)
    err = (y.double() - ref.double()).norm() / ref.double().norm()
    assert float(err) <= 2 * 2 ** 0.5 * STEP8 / 3 ** 0.5


def test_empty_and_leading_dimensions(K):
    x, xs, w, ws = operands(12, 256, 64)
    assert K.out_proj_fp8(x[:0], xs[:0], w, ws).shape == (0, 64)
    y = K.out_proj_fp8(x.view(3, 4, 256), xs.view(3, 4, 2), w, ws)
    assert y.shape == (3, 4, 64) and torch.equal(y.view(12, 64), K.out_proj_fp8(x, xs, w, ws))
    x8, sc = K.quant_fp8(torch.zeros(0, 256, device="cuda"))
    assert x8.shape == (0, 256) and sc.shape == (0, 2)
    x8, sc = K.norm_gate_fp8(*(torch.zeros(2, 0, 3, 64, device="cuda"),) * 2)
    assert x8.shape == (2, 0, 192) and sc.shape == (2, 0, 2)


def test_captured_and_on_another_stream(K):
    g = gen(5)
    o, gate = randn(g, 40, 4, 128, dtype=BF16), randn(g, 40, 4, 128, dtype=BF16)
    W8, Ws = K.quant_fp8(randn(g, 256, 512, std=0.05), 128)
    fn = lambda: K.out_proj_fp8(*K.norm_gate_fp8(o, gate), W8, Ws)
    graph, y = captured(fn)
    o.mul_(0.5).add_(0.1)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e = fn()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(e, y)


def test_refusals(K):
    x, xs, w, ws = operands(4, 256, 64)
    for bad in ((x.float(), xs, w, ws), (x, xs.double(), w, ws), (x, xs, w.view(torch.uint8), ws)):
        with pytest.raises(TypeError):
            K.out_proj_fp8(*bad)
    for bad in ((x, xs[:, :1].contiguous(), w, ws), (x, xs, w, ws.expand(2, 2).contiguous()), (x[:, :128], xs, w, ws),
                (x, xs.cpu(), w, ws)):
        with pytest.raises(ValueError):
            K.out_proj_fp8(*bad)
    with pytest.raises(TypeError):
        K.out_proj_fp8(x, xs, w, ws, out_dtype=torch.float16)
    with pytest.raises(K.KDAError):
        K.quant_fp8(torch.zeros(4, 256, device="cuda"), 64)
    with pytest.raises(TypeError):
        K.quant_fp8(torch.zeros(4, 256, device="cuda", dtype=torch.float16))
    with pytest.raises(K.KDAError):
        K.norm_gate_fp8(*(torch.zeros(2, 2, 64, device="cuda"),) * 2, eps=float("inf"))

"""The operators around the gated delta rule on tensors of more than 2^31 elements: offsets that pass 32 bits.  Each test
looks at the ends of the tensors, against a call on those parts alone."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import gen, randn, unit  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    yield K
    torch.cuda.empty_cache()


def test_states_far_into_the_pool(K):
    H, D, slots = 32, 128, (1 << 31) // (32 * 128 * 128) + 8
    pool = torch.empty(slots, H, D, D, device="cuda")
    g = gen(1)
    at = torch.tensor([slots - 1, 2, slots - 5], dtype=torch.int32, device="cuda")
    small = randn(g, 3, H, D, D)
    pool[at.long()] = small
    a = [unit(g, 3, 2, H, D, dtype=BF16), unit(g, 3, 2, H, D, dtype=BF16), randn(g, 3, 2, H, D, dtype=BF16),
         torch.rand((3, 2, H), generator=g, device="cuda").to(BF16)]
    z = randn(g, 3, 2, H, dtype=BF16)
    o = K.gdn_decode_step(*a, pool, z=z, slots=at)
    want = K.gdn_decode_step(*a, small, z=z)
    assert torch.equal(o, want) and torch.equal(pool[at.long()], small)


@pytest.mark.parametrize("D", [128, 70])  # whole vectors, and not
def test_token_rows_far_apart(K, D):
    S, H, stride = 3, 2, (1 << 30) + 64 * D
    base = torch.empty(2 * stride + H * D, dtype=BF16, device="cuda")
    q = base.as_strided((1, S, H, D), (0, stride, D, 1))
    near = randn(gen(2), 1, S, H, D, dtype=BF16)
    q.copy_(near)
    dq = randn(gen(3), 1, S, H, D)
    for x, y in zip(K.qk_norm(q, near, norm="rms"), K.qk_norm(near, near, norm="rms")):
        assert torch.equal(x, y)
    far, close = K.qk_norm_bwd(q, near, dq, dq, norm="rms"), K.qk_norm_bwd(near, near, dq, dq, norm="rms")
    assert torch.equal(far["dq"], close["dq"]) and torch.equal(far["dk"], close["dk"])


def test_rows_of_the_output_path(K):
    N, H, D = (1 << 31) // 4096 + 1000, 32, 128
    o = torch.zeros(N, H, D, dtype=BF16, device="cuda")
    gate = torch.zeros(N, H, D, dtype=BF16, device="cuda")
    ends = torch.cat([torch.arange(5), torch.arange(N - 5, N)]).cuda()
    o[ends], gate[ends] = randn(gen(4), 10, H, D, dtype=BF16), randn(gen(5), 10, H, D, dtype=BF16)
    x8, sc = K.norm_gate_fp8(o, gate)
    y8, ys = K.quant_fp8(o.view(N, H * D))
    e8, es = K.norm_gate_fp8(o[ends].contiguous(), gate[ends].contiguous())
    f8, fs = K.quant_fp8(o[ends].view(10, H * D).contiguous())
    b = lambda t: t.view(torch.uint8)
    assert torch.equal(b(x8)[ends], b(e8)) and torch.equal(sc[ends], es)
    assert torch.equal(b(y8)[ends], b(f8)) and torch.equal(ys[ends], fs)
    del o, gate, y8, ys
    for M in (4096, 4098):  # whole output vectors, and not
        W = K.quant_fp8(randn(gen(6), M, H * D, std=0.02), 128)
        y = K.out_proj_fp8(x8, sc, *W)
        part = K.out_proj_fp8(e8, es, *W)
        # another number of rows, another kernel: the blocks of the sum are added in another order
        assert float((y[ends].double() - part.double()).norm() / part.double().norm()) <= 2.0 ** -8
        del y


def test_gradients_of_a_very_long_sequence(K):
    """64 * 116,000 tokens of one head: a workspace of more than 2^31 floats.  No state outlasts two chunks at this decay
    (64 tokens: below e^-100), so the ends equal those of short sequences."""
    S, D, n, keep = 64 * 116000, 16, 512, 256
    g = gen(7)
    q, k = unit(g, 1, S, 1, D, dtype=BF16), unit(g, 1, S, 1, D, dtype=BF16)
    v, do = randn(g, 1, S, 1, D, dtype=BF16), randn(g, 1, S, 1, D, dtype=BF16)
    beta, z = torch.rand((1, S, 1), generator=g, device="cuda").to(BF16), randn(g, 1, S, 1, dtype=BF16)
    got = K.gdn_chunk_bwd(q, k, v, beta, do, z=z, g_min=-10.0)
    for part, cut in ((slice(0, n), slice(0, keep)), (slice(S - n, S), slice(n - keep, n))):
        short = K.gdn_chunk_bwd(*(t[:, part].contiguous() for t in (q, k, v, beta, do)), z=z[:, part].contiguous(),
                                g_min=-10.0)
        for name in ("dq", "dk", "dv", "dbeta", "dz"):
            x, y = got[name][:, part][:, cut], short[name][:, cut]
            assert float((x.double() - y.double()).abs().max()) <= 2.0 ** -15 * float(y.abs().max()), name

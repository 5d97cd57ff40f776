"""qk_norm and qk_norm_bwd against their formulas in 64 bits: types, head
layouts, head sizes that fill no vector, views of a fused projection's rows,
positions far out, gradients against the formula and against differences."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import U32, Guarded, assert_within, captured, gen, half_step, randn  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def turn(y, R, inter, pos, inv, sign=1.0):
    """The first R channels turned by sign * pos * inv, in 64 bits."""
    if not R:
        return y
    ang = sign * pos.double()[..., None, None] * inv.double()
    c, s = ang.cos(), ang.sin()
    out = y.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if inter else (slice(0, R // 2), slice(R // 2, R))
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def forward64(x, w, norm, eps, R, inter, pos, inv):
    x = x.double()
    n = x.square().sum(-1, keepdim=True) if norm == "l2" else x.square().mean(-1, keepdim=True)
    y = x / (n + eps).sqrt()
    y = y if w is None else y * w.double()
    return turn(y, R, inter, pos, inv)


def make(B, S, Hq, Hk, D, R, weight, fused, dtype, seed=0, max_pos=5000, offset=0):
    g = gen(seed)
    if fused:
        rows = randn(g, B, S, (Hq + Hk) * D + 5 * offset + 8, dtype=dtype)
        q = rows[..., offset:offset + Hq * D].unflatten(-1, (Hq, D))
        k = rows[..., offset + Hq * D:offset + (Hq + Hk) * D].unflatten(-1, (Hk, D))
    else:
        q, k = randn(g, B, S, Hq, D, dtype=dtype), randn(g, B, S, Hk, D, dtype=dtype)
    qw, kw = (1 + randn(g, D, std=0.2), 1 + randn(g, D, std=0.2)) if weight else (None, None)
    pos = inv = None
    if R:
        pos = torch.randint(-max_pos, max_pos, (B, S), generator=g, device="cuda")
        inv = (10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)).float()
    return q, k, qw, kw, pos, inv


# sums of D <= 256 squares, a reciprocal root (2 steps), three products and the turn: under 64 half-steps of fp32
# relative to the row's largest value (the turn mixes two channels), and one rounding to the output type
def tolerance(want, dtype):
    big = want.abs().amax(-1, keepdim=True)
    return half_step(dtype) * want.abs() * (1 + 2 ** -7) + 64 * U32 * big


CASES = [
    # B, S, Hq, Hk, D, R, interleaved, norm, weight, fused, dtype
    (1, 1, 1, 1, 128, 128, False, "rms", True, False, BF16),
    (2, 37, 8, 2, 128, 64, False, "rms", True, True, BF16),
    (1, 300, 16, 16, 128, 0, False, "l2", False, True, BF16),
    (3, 5, 3, 1, 64, 64, True, "l2", False, False, BF16),
    (1, 33, 5, 5, 256, 128, False, "rms", True, False, BF16),
    (1, 33, 5, 5, 256, 256, False, "rms", True, False, F32),
    (2, 9, 6, 3, 192, 192, False, "l2", True, True, F32),
    (2, 9, 6, 3, 192, 96, True, "l2", True, True, BF16),
    (1, 50, 7, 2, 32, 32, False, "rms", False, False, F32),
    (1, 50, 7, 2, 32, 16, False, "rms", False, False, BF16),
    (1, 21, 2, 2, 80, 80, False, "rms", True, False, BF16),
    (1, 21, 2, 2, 80, 40, False, "rms", True, False, BF16),      # halves of 20 channels: no whole vectors
    (2, 11, 4, 2, 100, 50, False, "l2", True, True, BF16),       # halves of 25 channels
    (2, 11, 4, 2, 7, 6, True, "rms", True, True, F32),
    (1, 3, 2, 1, 1, 0, False, "rms", True, False, F32),
    (1, 4500, 9, 9, 128, 128, False, "rms", True, False, BF16),  # many heads of a token in one item
]


@pytest.mark.parametrize("B,S,Hq,Hk,D,R,inter,norm,weight,fused,dtype", CASES)
def test_forward_matches_the_formula(K, B, S, Hq, Hk, D, R, inter, norm, weight, fused, dtype):
    q, k, qw, kw, pos, inv = make(B, S, Hq, Hk, D, R, weight, fused, dtype, seed=D + S)
    gq, gk = Guarded(q.shape, dtype), Guarded(k.shape, dtype)
    yq, yk = K.qk_norm(q, k, norm=norm, eps=1e-6, q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv,
                       interleaved=inter, out_q=gq.t, out_k=gk.t)
    gq.check("q_out")
    gk.check("k_out")
    for name, x, w, y in (("q", q, qw, yq), ("k", k, kw, yk)):
        want = forward64(x, w, norm, 1e-6, R, inter, pos, inv)
        assert_within(y, want, tolerance(want, dtype), name)


@pytest.mark.parametrize("grad", ["same", "f32"])
@pytest.mark.parametrize("B,S,Hq,Hk,D,R,inter,norm,weight,fused,dtype", CASES)
def test_backward_matches_the_formula(K, B, S, Hq, Hk, D, R, inter, norm, weight, fused, dtype, grad):
    q, k, qw, kw, pos, inv = make(B, S, Hq, Hk, D, R, weight, fused, dtype, seed=D + S + 1)
    g = gen(3)
    gt = F32 if grad == "f32" else dtype
    dyq, dyk = randn(g, *q.shape, dtype=gt), randn(g, *k.shape, dtype=gt)
    kw_args = dict(norm=norm, eps=1e-6, q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv, interleaved=inter)
    got = K.qk_norm_bwd(q, k, dyq, dyk, **kw_args)
    again = K.qk_norm_bwd(q, k, dyq, dyk, **kw_args)
    for n in got:
        assert (got[n] is None) == (again[n] is None)
        assert got[n] is None or torch.equal(got[n], again[n]), f"{n}: another run, other bits"
    for x, w, dy, dx, dw in ((q, qw, dyq, got["dq"], got["dq_weight"]), (k, kw, dyk, got["dk"], got["dk_weight"])):
        x64 = x.double()
        n = x64.square().sum(-1, keepdim=True) / (1 if norm == "l2" else D)
        r = 1 / (n + 1e-6).sqrt()
        up = turn(dy.double(), R, inter, pos, inv, sign=-1.0)
        h = up if w is None else up * w.double()
        y = x64 * r
        want = r * (h - y * (h * y).sum(-1, keepdim=True) / (1 if norm == "l2" else D))
        # h - y (h . y): each part rounded in fp32, relative to the row's largest part
        part = (r * h).abs().amax(-1, keepdim=True) + (r * y * (h * y).abs().sum(-1, keepdim=True) /
                                                       (1 if norm == "l2" else D)).abs().amax(-1, keepdim=True)
        assert_within(dx, want, half_step(dtype) * want.abs() * (1 + 2 ** -7) + 64 * U32 * part, "dx")
        if w is None:
            assert dw is None
        else:
            # a sum over the rows of up * y: `up` itself is a cos + b sin, each product rounded, so a row's term is off
            # by half-steps of |(a, b)| |y| even where the two cancel; |(a, b)| <= 2 max |dy| of the row
            rows = B * S * x.shape[2]
            size = (2 * dy.double().abs().amax(-1, keepdim=True) if R else up.abs()) * y.abs()
            assert_within(dw, (up * y).sum((0, 1, 2)), (rows + 64) * U32 * size.sum((0, 1, 2)), "dw")


@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_gradients_against_differences(K, norm):
    """Central differences of the definition in 64 bits, along random directions of q and of its weight."""
    q, k, qw, kw, pos, inv = make(1, 3, 2, 1, 24, 16, True, False, F32, seed=9)
    g = gen(10)
    dyq, dyk = randn(g, *q.shape), randn(g, *k.shape)
    got = K.qk_norm_bwd(q, k, dyq, dyk, norm=norm, q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv)
    loss = lambda x, w: (forward64(x, w, norm, 1e-6, 16, False, pos, inv) * dyq.double()).sum()
    for _ in range(4):
        u, v = randn(g, *q.shape).double(), randn(g, 24).double()
        e = 1e-6  # the difference's own error: 1e-12 of third order, 1e-16 / 1e-6 of rounding
        num = (loss(q.double() + e * u, qw.double()) - loss(q.double() - e * u, qw.double())) / (2 * e)
        ana = (got["dq"].double() * u).sum()
        assert abs(num - ana) <= 1e-5 * (got["dq"].double() * u).abs().sum()
        num = (loss(q.double(), qw.double() + e * v) - loss(q.double(), qw.double() - e * v)) / (2 * e)
        ana = (got["dq_weight"].double() * v).sum()
        assert abs(num - ana) <= 1e-5 * (got["dq_weight"].double() * v).abs().sum()


@pytest.mark.parametrize("pos0", [0, 1 << 20, (1 << 31) - 40, -(1 << 31)])
def test_far_positions_keep_their_angle(K, pos0):
    """Angles of up to 2^31 radians: the turn stays exact to fp32 (a frequency of 1 turns fastest)."""
    q, k, _, _, _, inv = make(1, 32, 2, 2, 64, 64, False, False, F32, seed=4)
    pos = (pos0 + torch.arange(32, device="cuda"))[None]
    yq, _ = K.qk_norm(q, k, positions=pos, inv_freq=inv)
    want = forward64(q, None, "l2", 1e-6, 64, False, pos, inv)
    assert_within(yq, want, tolerance(want, F32), "far")


@pytest.mark.parametrize("offset", [1, 3])
def test_rows_that_start_off_a_vector(K, offset):
    q, k, qw, kw, pos, inv = make(2, 13, 3, 2, 128, 128, True, True, BF16, seed=2, offset=offset)
    assert q.data_ptr() % 16
    yq, yk = K.qk_norm(q, k, norm="rms", q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv)
    for x, w, y in ((q, qw, yq), (k, kw, yk)):
        want = forward64(x, w, "rms", 1e-6, 128, False, pos, inv)
        assert_within(y, want, tolerance(want, BF16))


def test_rows_with_zeros_and_extremes(K):
    """A row of zeros gives zeros (eps > 0); NaN and infinity stay in their row."""
    q, k, *_ = make(1, 6, 2, 2, 128, 0, False, False, F32, seed=1)
    q[0, 1, 0] = 0
    q[0, 2, 1, 5] = float("nan")
    q[0, 3, 0, 7] = 1e-30
    k[0, 4, 1] = 1e-12
    yq, yk = K.qk_norm(q, k, norm="l2", eps=1e-6)
    for x, y in ((q, yq), (k, yk)):
        want = forward64(x, None, "l2", 1e-6, 0, False, None, None)
        assert_within(y, want, tolerance(want.nan_to_num(0.0), F32))
    assert bool((yq[0, 1, 0] == 0).all()) and int(yq.isnan().sum()) == 128


def test_no_tokens(K):
    q, k, qw, kw, pos, inv = make(0, 4, 3, 2, 64, 64, True, False, BF16)
    yq, yk = K.qk_norm(q, k, q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv)
    assert yq.shape == q.shape and yk.shape == k.shape
    got = K.qk_norm_bwd(q, k, yq, yk, q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv)
    assert bool((got["dq_weight"] == 0).all()) and bool((got["dk_weight"] == 0).all())


def test_captured_and_on_another_stream(K):
    q, k, qw, kw, pos, inv = make(2, 40, 4, 2, 128, 128, True, False, BF16, seed=6)
    fn = lambda: K.qk_norm(q, k, norm="rms", q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv)
    bw = lambda: K.qk_norm_bwd(q, k, q, k, norm="rms", q_weight=qw, k_weight=kw, positions=pos, inv_freq=inv)
    g, (yq, yk) = captured(fn)
    gb, back = captured(bw)
    q.mul_(-0.5).add_(0.25)
    pos.add_(17)
    g.replay()
    gb.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eq, ek = fn()
        eb = bw()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(yq, eq) and torch.equal(yk, ek)
    for n in eb:
        assert torch.equal(eb[n], back[n]), n


def test_refusals(K):
    q, k, qw, kw, pos, inv = make(1, 4, 3, 2, 64, 64, True, False, BF16)
    with pytest.raises(ValueError):
        K.qk_norm(q, k, positions=pos)                              # no frequencies
    with pytest.raises(ValueError):
        K.qk_norm(q, k, positions=pos[:, :3].contiguous(), inv_freq=inv)
    with pytest.raises(ValueError):
        K.qk_norm(q.transpose(1, 2), k.transpose(1, 2))             # heads not contiguous
    with pytest.raises(TypeError):
        K.qk_norm(q, k.float())
    with pytest.raises(TypeError):
        K.qk_norm(q.half(), k.half())
    with pytest.raises(ValueError):
        K.qk_norm(q, k, norm="layer")
    with pytest.raises(K.KDAError):
        K.qk_norm(q, k, eps=-1.0)
    with pytest.raises(K.KDAError):
        K.qk_norm(q, k, out_q=q)                                    # in place
    with pytest.raises(TypeError):
        K.qk_norm_bwd(q, k, q.double(), k.double())
    big = torch.zeros(1, 2, 2, 258, dtype=BF16, device="cuda")
    with pytest.raises(K.KDAError):
        K.qk_norm(big, big)
    with pytest.raises(K.KDAError):
        K.qk_norm(q, k, positions=pos, inv_freq=torch.ones(40, device="cuda"))  # more than D channels

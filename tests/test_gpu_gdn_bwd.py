"""gdn_chunk_bwd against the gradient of the recurrence in 64 bits (reverse mode
through the token loop), against differences, and against the per-channel
backward with the same decay in every channel."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import Guarded, assert_within, captured, gen, randn, unit  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32

# A product leaves out less than 2^-21 of its magnitudes and its fp32 accumulation over up to 128 terms in 3 parts adds up
# to 48 half-steps of 2^-24; a gradient is at most 8 products deep within a chunk, and what comes from other chunks has
# decayed: 8 (2^-21 + 48 2^-24) < 2^-15 of the largest element.
REL = 2.0 ** -15


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def make(B, S, H, Dk, Dv, dtype, decay, g_min, state, seed=0):
    g = gen(seed)
    d = dict(q=unit(g, B, S, H, Dk, dtype=dtype), k=unit(g, B, S, H, Dk, dtype=dtype), v=randn(g, B, S, H, Dv, dtype=dtype),
             beta=torch.rand((B, S, H), generator=g, device="cuda").to(dtype), d_o=randn(g, B, S, H, Dv, dtype=dtype))
    z = randn(g, B, S, H, std=1.5)
    opt = dict(z=z.to(dtype)) if decay == "z" else dict(log_decay=g_min * torch.sigmoid(z) * 1.1)  # some clamped
    if state:
        opt["initial_state"] = randn(g, B, H, Dk, Dv, std=0.3)
        opt["d_final_state"] = randn(g, B, H, Dk, Dv, std=0.3)
    return d, opt


def forward64(q, k, v, beta, ld, s0):
    S, out = s0, []
    for t in range(q.shape[1]):
        D = ld[:, t].exp()[..., None, None] * S
        r = beta[:, t][..., None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", D, k[:, t]))
        S = D + k[:, t][..., :, None] * r[..., None, :]
        out.append(torch.einsum("bhkv,bhk->bhv", S, q[:, t]))
    return (torch.stack(out, 1) if out else v), S


def loss64(d, opt, g_min, x):
    ld = x["log"].clamp(g_min, 0.0) if "log_decay" in opt else g_min * torch.sigmoid(x["log"])
    o, sT = forward64(x["q"], x["k"], x["v"], x["beta"], ld, x["s0"])
    total = (o * d["d_o"].double()).sum()
    return total if opt.get("d_final_state") is None else total + (sT * opt["d_final_state"].double()).sum()


def leaves64(d, opt):
    B, _, H, Dk = d["q"].shape
    s0 = opt.get("initial_state")
    x = {n: d[n].double() for n in ("q", "k", "v", "beta")}
    x["log"] = (opt["z"] if "z" in opt else opt["log_decay"]).double()
    x["s0"] = torch.zeros(B, H, Dk, d["v"].shape[-1], dtype=torch.float64, device="cuda") if s0 is None else s0.double()
    return {n: t.clone().requires_grad_() for n, t in x.items()}


def gradients64(d, opt, g_min):
    x = leaves64(d, opt)
    g = torch.autograd.grad(loss64(d, opt, g_min, x), list(x.values()))
    return dict(zip(("dq", "dk", "dv", "dbeta", "dlog_decay" if "log_decay" in opt else "dz", "d_initial_state"), g))


def check(got, want, rel=REL):
    for n, w in want.items():
        assert got[n].dtype == F32
        assert_within(got[n], w, rel * float(w.abs().max()) if w.numel() else 0.0, n)


CASES = [
    # B, S, H, Dk, Dv, dtype, decay, g_min, state
    (1, 64, 1, 128, 128, BF16, "z", -5.0, True),
    (2, 130, 3, 128, 128, BF16, "z", -0.25, True),
    (1, 200, 2, 128, 128, F32, "log", -0.25, True),
    (1, 1, 2, 128, 128, BF16, "z", -5.0, True),
    (3, 63, 2, 64, 32, BF16, "log", -1.0, False),
    (2, 65, 1, 72, 100, F32, "log", -0.25, True),
    (1, 129, 2, 1, 1, F32, "z", -2.0, True),
    (2, 77, 2, 17, 128, BF16, "z", -20.0, True),
    (1, 150, 2, 128, 13, F32, "z", -60.0, False),
    (1, 400, 1, 32, 32, F32, "log", -0.02, True),   # almost no decay: everything is carried through seven chunks
]


@pytest.mark.parametrize("B,S,H,Dk,Dv,dtype,decay,g_min,state", CASES)
def test_matches_reverse_mode(K, B, S, H, Dk, Dv, dtype, decay, g_min, state):
    d, opt = make(B, S, H, Dk, Dv, dtype, decay, g_min, state, seed=S + Dk)
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=g_min, **opt)
    again = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=g_min, **opt)
    for n in got:
        assert torch.equal(got[n], again[n]), f"{n}: another run, other bits"
    check(got, gradients64(d, opt, g_min))


def test_repeated_and_opposite_keys(K):
    """The least benign system inside a chunk: every key +- the same direction, writes of full strength."""
    d, opt = make(1, 128, 2, 64, 64, F32, "log", -0.05, True, seed=5)
    d["k"] = (d["k"][:, :1] * torch.where(torch.arange(128, device="cuda") % 3 == 0, -1.0, 1.0)[None, :, None, None]).contiguous()
    d["beta"].fill_(1.0)
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=-0.05, **opt)
    check(got, gradients64(d, opt, -0.05))


def test_against_differences(K):
    """Central differences of the 64-bit loss along random directions of each input (third-order error 1e-10)."""
    d, opt = make(1, 70, 1, 16, 16, F32, "z", -1.0, True, seed=21)
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=-1.0, **opt)
    names = {"q": "dq", "k": "dk", "v": "dv", "beta": "dbeta", "log": "dz", "s0": "d_initial_state"}
    x = {n: t.detach() for n, t in leaves64(d, opt).items()}
    g, e = gen(22), 1e-5
    for n, out in names.items():
        u = randn(g, *x[n].shape).double()
        up, down = ({**x, n: x[n] + s * e * u} for s in (1, -1))
        num = (loss64(d, opt, -1.0, up) - loss64(d, opt, -1.0, down)) / (2 * e)
        ana = (got[out].double() * u).sum()
        assert abs(float(num - ana)) <= 2 * REL * float((got[out].double() * u).abs().sum()), n


def test_agrees_with_the_per_channel_backward(K):
    d, opt = make(2, 150, 2, 128, 128, BF16, "z", -5.0, True, seed=7)
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **opt)
    wide = dict(opt, z=opt["z"][..., None].expand(-1, -1, -1, 128).contiguous())
    ref = K.chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **wide)
    ref["dz"] = ref["dz"].double().sum(-1)
    for n in ref:
        err = (got[n].double() - ref[n].double()).norm() / ref[n].double().norm()
        assert float(err) <= 2e-4, n                      # the per-channel backward's own tolerance


def test_no_tokens_passes_the_state_gradient_through(K):
    d, opt = make(2, 0, 2, 32, 32, BF16, "z", -5.0, True)
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **opt)
    assert torch.equal(got["d_initial_state"], opt["d_final_state"]) and got["dq"].shape == (2, 0, 2, 32)
    del opt["d_final_state"]
    assert bool((K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **opt)["d_initial_state"] == 0).all())
    d, opt = make(0, 5, 2, 32, 32, BF16, "z", -5.0, True)
    assert K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **opt)["dk"].shape == (0, 5, 2, 32)


def test_a_non_finite_head_leaves_the_others(K):
    d, opt = make(2, 100, 3, 64, 64, F32, "z", -1.0, True, seed=3)
    clean = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=-1.0, **opt)
    d["v"][1, 70, 2, 3] = float("nan")
    got = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], g_min=-1.0, **opt)
    assert bool(got["dk"][1, :, 2].isnan().any())
    for n in ("dq", "dk", "dv"):
        assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][1, :, :2], clean[n][1, :, :2]), n


def test_writes_stay_inside(K):
    """Guard bands around every output and the workspace, through the C entry point."""
    import ctypes
    from kimi_delta_attention_21_b200 import _lib as L
    lib = K.load_library()
    for dtype, B, S, H, Dk, Dv in ((BF16, 2, 100, 3, 128, 128), (F32, 1, 65, 2, 33, 70)):
        d, opt = make(B, S, H, Dk, Dv, dtype, "z", -3.0, True, seed=1)
        out = {n: Guarded(s, F32) for n, s in (("dq", d["q"].shape), ("dk", d["k"].shape), ("dv", d["v"].shape),
                                               ("dbeta", (B, S, H)), ("dz", (B, S, H)),
                                               ("d_initial_state", (B, H, Dk, Dv)))}
        a = L.RecBwdArgs(B=B, S=S, H=H, D_k=Dk, D_v=Dv, dtype=L.KDA_BF16 if dtype == BF16 else L.KDA_F32, g_min=-3.0,
                         z=opt["z"].data_ptr(), initial_state=opt["initial_state"].data_ptr(),
                         d_final_state=opt["d_final_state"].data_ptr(), stream=torch.cuda.current_stream().cuda_stream,
                         **{n: t.data_ptr() for n, t in d.items()}, **{n: x.t.data_ptr() for n, x in out.items()})
        n = ctypes.c_size_t(0)
        assert lib.kda_gdn_chunk_bwd_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
        ws = Guarded((n.value,), torch.uint8)
        a.workspace, a.workspace_bytes = ws.t.data_ptr(), n.value
        assert lib.kda_gdn_chunk_bwd(ctypes.byref(a)) == 0
        ws.check("workspace")
        ref = K.gdn_chunk_bwd(*(d[m] for m in ("q", "k", "v", "beta", "d_o")), g_min=-3.0, **opt)
        for m, x in out.items():
            x.check(m)
            assert torch.equal(x.t, ref[m]), m


def test_unaligned_inputs(K):
    d, opt = make(1, 90, 2, 128, 128, BF16, "z", -5.0, True, seed=6)
    ref = K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **opt)
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)
    got = K.gdn_chunk_bwd(*(off(d[m]) for m in ("q", "k", "v", "beta", "d_o")), **{m: off(t) for m, t in opt.items()})
    for n in ref:
        assert torch.equal(got[n], ref[n]), n


def test_captured_and_on_another_stream(K):
    d, opt = make(2, 140, 2, 128, 128, BF16, "z", -5.0, True, seed=9)
    fn = lambda: K.gdn_chunk_bwd(d["q"], d["k"], d["v"], d["beta"], d["d_o"], **opt)
    g, got = captured(fn)
    d["v"].mul_(0.5)
    opt["z"].add_(0.25)
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ref = fn()
    torch.cuda.current_stream().wait_stream(side)
    for n in ref:
        assert torch.equal(got[n], ref[n]), n


def test_refusals(K):
    d, opt = make(1, 20, 2, 32, 32, BF16, "z", -5.0, True)
    args = [d[m] for m in ("q", "k", "v", "beta", "d_o")]
    with pytest.raises(ValueError):
        K.gdn_chunk_bwd(*args, z=d["q"])                       # per-channel decay
    with pytest.raises(K.KDAError):
        K.gdn_chunk_bwd(*args)                                 # no decay
    with pytest.raises(K.KDAError):
        K.gdn_chunk_bwd(*args, z=opt["z"], g_min=0.0)
    with pytest.raises(TypeError):
        K.gdn_chunk_bwd(args[0], args[1].float(), *args[2:], z=opt["z"])
    with pytest.raises(ValueError):
        K.gdn_chunk_bwd(*args[:4], args[4][:, :10], z=opt["z"])
    with pytest.raises(K.KDAError):
        K.gdn_chunk_bwd(*args, z=opt["z"], workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    big = torch.zeros(1, 2, 1, 129, dtype=BF16, device="cuda")
    with pytest.raises(K.KDAError):
        K.gdn_chunk_bwd(big, big, big, torch.zeros(1, 2, 1, dtype=BF16, device="cuda"), big,
                        z=torch.zeros(1, 2, 1, dtype=BF16, device="cuda"))

"""gdn_decode_step against the recurrence in 64 bits: one and several tokens,
states in a pool, padded rows, odd head sizes, the chunked prefill's own
continuation, captured and on another stream."""
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import U32, Guarded, assert_within, captured, gen, half_step, randn, unit  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def make(B, T, H, Dk, Dv, dtype, n, decay, g_min, gate, seed=0):
    g = gen(seed)
    d = dict(q=unit(g, B, T, H, Dk, dtype=dtype), k=unit(g, B, T, H, Dk, dtype=dtype), v=randn(g, B, T, H, Dv, dtype=dtype),
             beta=torch.rand((B, T, H), generator=g, device="cuda").to(dtype), z=None, log_decay=None, gate_logits=None)
    z = randn(g, B, T, H)
    if decay == "z":
        d["z"] = z.to(dtype)
    else:
        d["log_decay"] = g_min * torch.sigmoid(z) * 1.2  # some below g_min: clamped
    if gate:
        d["gate_logits"] = randn(g, B, T, H, Dv, dtype=dtype)
    return d, randn(g, n, H, Dk, Dv, std=0.1)


def recurrence64(d, state, g_min, rows, eps=1e-6):
    """(o~ or gated o, updated pool, a bound of |o~|'s size) in 64 bits; rows: the state of each sequence, < 0: skipped."""
    x = {n: (None if t is None else t.double()) for n, t in d.items()}
    ld = x["log_decay"].clamp(g_min, 0.0) if x["z"] is None else g_min * torch.sigmoid(x["z"])
    live = [i for i, r in enumerate(rows) if r >= 0]
    at = torch.tensor([rows[i] for i in live], device=state.device, dtype=torch.long)
    pool = state.double().clone()
    S = pool[at]
    out = []
    for t in range(d["q"].shape[1]):
        q, k, v = (x[n][live, t] for n in ("q", "k", "v"))
        S = ld[live, t].exp()[..., None, None] * S
        r = x["beta"][live, t][..., None] * (v - torch.einsum("bhkv,bhk->bhv", S, k))
        S = S + k[..., :, None] * r[..., None, :]
        out.append(torch.einsum("bhkv,bhk->bhv", S, q))
    pool[at] = S
    core = torch.stack(out, 1) if out else x["v"][live][:, :0]
    o = core
    if x["gate_logits"] is not None:
        o = core / (core.square().mean(-1, keepdim=True) + eps).sqrt() * torch.sigmoid(x["gate_logits"][live])
    return live, o, core, pool


def check(d, state0, state, o, g_min, rows, dtype, T):
    live, want, core, pool = recurrence64(d, state0, g_min, rows)
    # a step sums D_k products twice and rounds each state element four times, relative to the largest of the states and
    # values (|k| = |q| = 1): under 16 half-steps a token, and the errors of earlier tokens are carried on
    size = max(float(state0.abs().max()), float(d["v"].double().abs().max()), 1.0)
    err = 16 * max(T, 1) * U32 * size
    assert_within(state, pool, err, "state")
    if d["gate_logits"] is not None:  # the norm divides by the row's own size
        rms = (core.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        err = err * 2 / rms + 16 * U32 * want.abs()
    assert_within(o[live], want, half_step(dtype) * want.abs() * (1 + 2 ** -7) + err, "o")


CASES = [
    # B, T, H, Dk, Dv, dtype, decay, g_min, gate
    (1, 1, 1, 128, 128, BF16, "z", -5.0, True),
    (5, 1, 3, 128, 128, BF16, "log", -1.0, False),
    (3, 7, 2, 128, 128, BF16, "z", -5.0, True),
    (2, 33, 2, 128, 128, F32, "z", -0.1, True),
    (4, 2, 2, 128, 128, F32, "log", -20.0, False),
    (3, 4, 5, 96, 72, F32, "log", -1.0, False),
    (2, 3, 2, 1, 1, F32, "z", -5.0, True),
    (2, 3, 2, 7, 128, BF16, "z", -5.0, True),
    (2, 5, 3, 128, 33, BF16, "z", -60.0, True),
    (300, 1, 2, 64, 64, BF16, "z", -5.0, False),
]


@pytest.mark.parametrize("B,T,H,Dk,Dv,dtype,decay,g_min,gate", CASES)
def test_matches_the_recurrence(K, B, T, H, Dk, Dv, dtype, decay, g_min, gate):
    d, state0 = make(B, T, H, Dk, Dv, dtype, B, decay, g_min, gate, seed=B + T)
    gs, go = Guarded(state0.shape, F32), Guarded(d["v"].shape, dtype)
    gs.t.copy_(state0)
    K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], gs.t, z=d["z"], log_decay=d["log_decay"], g_min=g_min,
                      gate_logits=d["gate_logits"], out=go.t)
    gs.check("state")
    go.check("o")
    check(d, state0, gs.t, go.t, g_min, list(range(B)), dtype, T)


@pytest.mark.parametrize("T,D,dtype", [(1, 128, BF16), (3, 128, F32), (2, 40, BF16)])
def test_slots_padding_and_bad_slots(K, T, D, dtype):
    """States by slot; padded rows untouched; a slot outside the pool or given twice is skipped and reported."""
    B, H, n = 9, 2, 12
    d, state0 = make(B, T, H, D, D, dtype, n, "z", -2.0, False, seed=T)
    rows = [7, -1, 3, 11, 0, 3, 12, -5, 5]
    eff = [7, -1, 3, 11, 0, -1, -1, -1, 5]      # the second 3, and 12, are skipped
    state, o = state0.clone(), torch.full_like(d["v"], 2.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], state, z=d["z"], g_min=-2.0, out=o, dev_status=status,
                      slots=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    assert int(status) == 1
    check(d, state0, state, o, -2.0, eff, dtype, T)
    for i, r in enumerate(eff):
        if r < 0:
            assert bool((o[i] == 2.5).all())
    untouched = [i for i in range(n) if i not in eff]
    assert torch.equal(state[untouched], state0[untouched])
    status.zero_()
    good = torch.tensor(eff[:5] + [-1, 8, -1, 5], dtype=torch.int32, device="cuda")
    K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], state, z=d["z"], g_min=-2.0, dev_status=status, slots=good)
    assert int(status) == 0


@pytest.mark.parametrize("Dk,Dv", [(32, 32), (33, 128), (16, 15), (64, 128), (65, 20), (8, 4), (31, 96), (63, 31)])
@pytest.mark.parametrize("T,dtype", [(1, BF16), (5, F32)])
def test_matches_the_recurrence_for_few_key_channels(K, T, Dk, Dv, dtype):
    test_matches_the_recurrence(K, 9, T, 3, Dk, Dv, dtype, "z", -5.0, True)


def test_tokens_at_once_equal_tokens_one_by_one(K):
    d, state0 = make(4, 6, 3, 128, 128, BF16, 4, "z", -3.0, True, seed=8)
    all_at_once, one = state0.clone(), state0.clone()
    o = K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], all_at_once, z=d["z"], gate_logits=d["gate_logits"])
    for t in range(6):
        at = lambda n: d[n][:, t].contiguous()
        ot = K.gdn_decode_step(at("q"), at("k"), at("v"), at("beta"), one, z=at("z"), gate_logits=at("gate_logits"))
        assert torch.equal(ot, o[:, t])
    assert torch.equal(one, all_at_once)


def test_continues_a_chunked_prefill(K):
    """The prefill's final state, then tokens one by one, against the recurrence over all of them."""
    d, state0 = make(2, 140, 3, 128, 128, BF16, 2, "z", -5.0, False, seed=12)
    cut = lambda a, b: {n: None if t is None else t[:, a:b].contiguous() for n, t in d.items()}
    p, r = cut(0, 130), cut(130, 140)
    _, sf = K.gdn_chunk_fwd(p["q"], p["k"], p["v"], p["beta"], z=p["z"], initial_state=state0)
    start = sf.clone()
    o = K.gdn_decode_step(r["q"], r["k"], r["v"], r["beta"], sf, z=r["z"])
    check(r, start, sf, o, -5.0, [0, 1], BF16, 10)
    _, want, _, pool = recurrence64(d, state0, -5.0, [0, 1])
    assert float((o.double() - want[:, 130:]).abs().max()) <= 2e-2     # the chunk engine's own bound
    assert float((sf.double() - pool).norm() / pool.norm()) <= 1e-2


def test_non_finite_values_stay_in_their_state(K):
    d, state0 = make(3, 2, 2, 128, 128, F32, 3, "z", -5.0, False, seed=3)
    d["v"][1, 0, 0, 5] = float("inf")
    state0[2, 1, 4, 4] = float("nan")
    state = state0.clone()
    o = K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], state, z=d["z"])
    assert bool(state[0].isfinite().all()) and bool(o[0].isfinite().all())
    assert bool(state[1, 1].isfinite().all()) and bool(state[2, 0].isfinite().all())
    assert not bool(state[1, 0, :, 5].isfinite().any()) and bool(state[2, 1, :, 4].isnan().all())
    keep = [c for c in range(128) if c != 5]
    assert bool(state[1, 0][:, keep].isfinite().all())


def test_empty_calls(K):
    d, state0 = make(2, 0, 2, 64, 64, BF16, 2, "z", -5.0, False)
    state = state0.clone()
    assert K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], state, z=d["z"]).shape == (2, 0, 2, 64)
    d, _ = make(0, 1, 2, 64, 64, BF16, 2, "z", -5.0, False)
    K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], state, z=d["z"])
    assert torch.equal(state, state0)


def test_unaligned_state_and_vectors(K):
    d, state0 = make(2, 2, 2, 128, 128, BF16, 2, "z", -5.0, True, seed=4)
    gs = Guarded(state0.shape, F32, offset=1)
    gs.t.copy_(state0)
    off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)
    o = K.gdn_decode_step(off(d["q"]), off(d["k"]), off(d["v"]), off(d["beta"]), gs.t, z=off(d["z"]),
                          gate_logits=off(d["gate_logits"]))
    gs.check()
    check(d, state0, gs.t, o, -5.0, [0, 1], BF16, 2)


def test_captured_and_on_another_stream(K):
    d, state0 = make(6, 1, 4, 128, 128, BF16, 8, "z", -5.0, True, seed=5)
    slots = torch.tensor([5, 2, 0, -1, 7, 1], dtype=torch.int32, device="cuda")
    state = state0.clone()
    fn = lambda: K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], state, z=d["z"], gate_logits=d["gate_logits"],
                                   slots=slots)
    g, o = captured(fn)
    state.copy_(state0)
    slots.copy_(torch.tensor([1, -1, 0, 6, 4, 3], dtype=torch.int32, device="cuda"))
    for _ in range(3):
        g.replay()
    mine = state0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            eo = K.gdn_decode_step(d["q"], d["k"], d["v"], d["beta"], mine, z=d["z"], gate_logits=d["gate_logits"],
                                   slots=slots)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(mine, state)
    live = [0, 2, 3, 4, 5]
    assert torch.equal(eo[live], o[live])


def test_refusals(K):
    d, state = make(2, 1, 2, 64, 64, BF16, 2, "z", -5.0, False)
    args = (d["q"], d["k"], d["v"], d["beta"])
    with pytest.raises(K.KDAError):
        K.gdn_decode_step(*args, state)                                        # no decay
    with pytest.raises(K.KDAError):
        K.gdn_decode_step(*args, state, z=d["z"], g_min=1.0)
    with pytest.raises(K.KDAError):
        K.gdn_decode_step(*args, state[:1], z=d["z"])                          # two sequences, one state
    with pytest.raises(TypeError):
        K.gdn_decode_step(*args, state.half(), z=d["z"])
    with pytest.raises(TypeError):
        K.gdn_decode_step(*args, state, z=d["z"], slots=torch.tensor([0, 1], device="cuda"))
    with pytest.raises(ValueError):
        K.gdn_decode_step(*args, state, z=d["z"], slots=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        K.gdn_decode_step(d["q"][..., ::2], *args[1:], state, z=d["z"])
    with pytest.raises(ValueError):
        K.gdn_decode_step(*args, state, z=d["z"].cpu())

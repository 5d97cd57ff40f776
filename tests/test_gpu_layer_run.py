"""The operators around the gated delta rule one after the other, as a layer uses them: serving (prefill, decode from a
pool of states, the e4m3 output), training (gradients to the raw projections), one captured decode step, two streams at
once, and the bounds-checked build."""
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
from layer_testlib import captured, gen, randn  # noqa: E402
from test_gpu_gdn_bwd import forward64  # noqa: E402
from test_gpu_qk_norm import forward64 as norm64  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def K():
    import kimi_delta_attention_21_b200 as K
    K.load_library()
    return K


def raw(B, S, H, D, dtype, seed):
    """What a layer's projections give: rows of queries, keys and values, write strengths, decay logits, output gate."""
    g = gen(seed)
    rows = randn(g, B, S, 3 * H * D, dtype=dtype)
    q, k, v = (rows[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in range(3))
    beta = torch.rand((B, S, H), generator=g, device="cuda").to(dtype)
    z, gate = randn(g, B, S, H, dtype=dtype), randn(g, B, S, H, D, dtype=dtype)
    pos = (torch.arange(S, device="cuda") + torch.tensor([[0], [70000], [1 << 20]], device="cuda")[:B]).contiguous()
    inv = (10000.0 ** (-torch.arange(0, 64, 2, device="cuda").double() / 64)).float()
    return q, k, v.contiguous(), beta, z, gate, pos, inv


def test_serving_prefill_then_decode(K):
    B, S, T, H, D, Dm = 3, 150, 20, 4, 128, 512   # 130 tokens at once, 17 one by one, 3 drafted together
    q, k, v, beta, z, gate, pos, inv = raw(B, S, H, D, BF16, 1)
    W = randn(gen(2), Dm, H * D, std=(H * D) ** -0.5)
    W8, Ws = K.quant_fp8(W, 128)
    turn = dict(inv_freq=inv)
    at = lambda t, a, b: t[:, a:b].contiguous()
    P = S - T
    qn, kn = K.qk_norm(q[:, :P], k[:, :P], positions=at(pos, 0, P), **turn)
    o, sf = K.gdn_chunk_fwd(qn, kn, at(v, 0, P), at(beta, 0, P), z=at(z, 0, P))
    pool = torch.zeros(7, H, D, D, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()] = sf
    xs = [K.norm_gate_fp8(o, at(gate, 0, P))]
    steps = [(t, t + 1) for t in range(P, S - 3)] + [(S - 3, S)]
    for a, b in steps:
        qn, kn = K.qk_norm(q[:, a:b], k[:, a:b], positions=at(pos, a, b), **turn)
        o = K.gdn_decode_step(qn, kn, at(v, a, b), at(beta, a, b), pool, z=at(z, a, b), slots=slots)
        xs.append(K.norm_gate_fp8(o, at(gate, a, b)))
    y = torch.cat([K.out_proj_fp8(x8, sc, W8, Ws) for x8, sc in xs], 1)
    # the same layer in 64 bits
    q64, k64 = (norm64(x, None, "l2", 1e-6, 64, False, pos, inv) for x in (q, k))
    core, state = forward64(q64, k64, v.double(), beta.double(), -5.0 * torch.sigmoid(z.double()),
                            torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda"))
    x = core / (core.square().mean(-1, keepdim=True) + 1e-6).sqrt() * torch.sigmoid(gate.double())
    want = x.flatten(2) @ W.double().mT
    # the two e4m3 factors are off by a random half-step each (2^-4 / sqrt(3) of the value); the bf16 queries, keys and
    # chunk engine by less than half of that
    assert float((y.double() - want).norm() / want.norm()) <= 1.5 * 2 ** 0.5 * 2 ** -4 / 3 ** 0.5
    assert float((pool[slots.long()].double() - state).norm() / state.norm()) <= 1e-2
    untouched = [i for i in range(7) if i not in (0, 4, 6)]
    assert bool((pool[untouched] == 0).all())


def test_training_gradients_to_the_raw_projections(K):
    B, S, H, D = 2, 140, 3, 64
    q, k, v, beta, z, _, pos, inv = raw(B, S, H, D, F32, 3)
    g = gen(4)
    s0, d_o = randn(g, B, H, D, D, std=0.1), randn(g, B, S, H, D)
    w = D ** -0.5 * (1 + randn(g, D, std=0.1))       # unit keys from the RMS norm: the weight carries 1 / sqrt(D)
    kw = dict(norm="rms", q_weight=w, k_weight=w, positions=pos, inv_freq=inv)
    qn, kn = K.qk_norm(q, k, **kw)
    core = K.gdn_chunk_bwd(qn, kn, v, beta, d_o, z=z, g_min=-1.0, initial_state=s0)
    front = K.qk_norm_bwd(q, k, core["dq"], core["dk"], **kw)
    x = {n: t.double().clone().requires_grad_() for n, t in dict(q=q, k=k, v=v, beta=beta, z=z, s0=s0, qw=kw["q_weight"],
                                                                 kw=kw["k_weight"]).items()}
    o, _ = forward64(norm64(x["q"], x["qw"], "rms", 1e-6, 64, False, pos, inv),
                     norm64(x["k"], x["kw"], "rms", 1e-6, 64, False, pos, inv), x["v"], x["beta"],
                     -1.0 * torch.sigmoid(x["z"]), x["s0"])
    grads = dict(zip(x, torch.autograd.grad((o * d_o.double()).sum(), list(x.values()))))
    got = dict(q=front["dq"], k=front["dk"], v=core["dv"], beta=core["dbeta"], z=core["dz"], s0=core["d_initial_state"],
               qw=front["dq_weight"], kw=front["dk_weight"])
    # the core's 2^-15 of the largest element, once more through the norm's backward (fp32): under 2^-14
    for n, want in grads.items():
        assert float((got[n].double() - want).abs().max()) <= 2.0 ** -14 * float(want.abs().max()), n


def test_one_captured_decode_step(K):
    B, H, D, Dm = 5, 4, 128, 256
    q, k, v, beta, z, gate, _, inv = raw(1, B, H, D, BF16, 5)
    q, k, v, beta, z, gate = (t[0] for t in (q, k, v, beta, z, gate))
    pos = torch.randint(0, 1 << 20, (B,), generator=gen(6), device="cuda")
    W8, Ws = K.quant_fp8(randn(gen(7), Dm, H * D, std=0.05), 128)
    slots = torch.tensor([2, -1, 0, 5, 1], dtype=torch.int32, device="cuda")
    first = randn(gen(8), 6, H, D, D, std=0.1)
    out = torch.zeros(B, H, D, dtype=BF16, device="cuda")

    def step(pool):
        qn, kn = K.qk_norm(q, k, positions=pos, inv_freq=inv)
        o = K.gdn_decode_step(qn, kn, v, beta, pool, z=z, slots=slots, out=out)
        return K.out_proj_fp8(*K.norm_gate_fp8(o, gate), W8, Ws)

    pool = first.clone()
    graph, y = captured(lambda: step(pool))
    pool.copy_(first)
    mine = first.clone()
    for i in range(3):
        pos.add_(1)
        v.mul_(0.9)
        slots.copy_(slots.roll(1))
        graph.replay()
        got = y.clone()
        assert torch.equal(got, step(mine)), i
    assert torch.equal(pool, mine)


def test_two_streams_at_once(K):
    """The same operators on two streams, each with its own buffers: the results of one after the other."""
    def work(seed):
        q, k, v, beta, z, gate, pos, inv = raw(2, 300, 4, 128, BF16, seed)
        qn, kn = K.qk_norm(q, k, norm="rms", q_weight=inv.new_ones(128), k_weight=inv.new_ones(128))
        back = K.gdn_chunk_bwd(qn, kn, v, beta, gate, z=z)
        front = K.qk_norm_bwd(q, k, back["dq"], back["dk"], norm="rms", q_weight=inv.new_ones(128),
                              k_weight=inv.new_ones(128))
        x8, sc = K.norm_gate_fp8(v, gate)
        y = K.out_proj_fp8(x8, sc, *K.quant_fp8(randn(gen(seed), 640, 512, std=0.05), 128))
        return [*back.values(), *front.values(), y]

    alone = [work(11), work(12)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    together = [None, None]
    for _ in range(2):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                together[i] = work(11 + i)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_gradients_of_two_graphs_and_two_streams(K):
    """Two captured gradient passes with workspaces of their own, replayed at once on two streams, against eager calls."""
    def inputs(seed, B, S, H, D, dtype):
        q, k, v, beta, z, _, _, _ = raw(B, S, H, D, dtype, seed)
        qn, kn = K.qk_norm(q, k)
        return (qn, kn, v, beta, randn(gen(seed + 50), B, S, H, D, dtype=dtype)), dict(z=z, g_min=-3.0)
    jobs = [inputs(21, 1, 700, 3, 128, BF16), inputs(22, 2, 130, 2, 64, F32)]
    want = [K.gdn_chunk_bwd(*a, **kw) for a, kw in jobs]
    graphs, got = [], []
    for a, kw in jobs:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            K.gdn_chunk_bwd(*a, **kw)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(K.gdn_chunk_bwd(*a, **kw))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, r in zip(want, got):  # nothing is added in a varying order: the same bits
        for n in w:
            assert w[n] is None and r[n] is None or torch.equal(w[n], r[n]), n


def test_checked_build_runs_clean_and_matches(tmp_path):
    out = tmp_path / "checked.npz"
    env = dict(os.environ, KDA_LIBRARY="libkda_checked.so")
    r = subprocess.run([sys.executable, os.path.join(HERE, "layer_checked_cases.py"), str(out)], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    got = np.load(out)
    assert int(got["_checked_build"]) == 1 and int(got["_bounds_errors"]) == 0
    import layer_checked_cases
    want, counters = layer_checked_cases.run_cases()
    assert counters == {"bounds_errors": 0, "checked_build": 0}
    assert set(want) == {n for n in got.files if not n.startswith("_")}
    for n, x in want.items():
        assert np.array_equal(got[n], x, equal_nan=True), f"{n}: checked and normal builds differ"

"""Measured cases of the operators around the gated delta rule layer.

Six operators, one per ``op`` of a case, in the order a layer runs them:

* ``qk_norm``        per-head norm of queries and keys (L2, or RMS with a weight), with the rotation by position
* ``qk_norm_bwd``    its gradients (queries, keys, and the two weights)
* ``gdn_decode``     the gated delta rule token by token from a pool of states, advanced in place
* ``gdn_bwd``        the gradients of the gated delta rule over whole sequences
* ``norm_gate_fp8``  the per-head output norm and gate, quantised to e4m3 with one scale per 128 channels
* ``out_proj_fp8``   the output projection from e4m3 operands (activations 1 x 128, weights 128 x 128)

``run`` computes a case in plain torch operations, or, with ``own`` set, by the framework's entry points.
``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest normal fp32 value: no scale is below it
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 256 sequences at 32 heads: RMS norm with a weight and the rotation at positions far apart
        dict(name="qk_norm_decode_256", op="qk_norm", B=256, S=1, Hq=32, Hk=32, D=128, R=128, interleaved=False,
             norm="rms", weight=True, fused=True, dtype="bf16", max_pos=1 << 20),
        # the L2 norm in front of a prefill of 4096 tokens, 16 heads, read from the fused projection's rows
        dict(name="qk_norm_prefill_4k", op="qk_norm", B=1, S=4096, Hq=16, Hk=16, D=128, R=0, interleaved=False,
             norm="l2", weight=False, fused=True, dtype="bf16", max_pos=0),
        # a training batch of 8 x 2048 tokens: RMS norm, weights and rotation, fp32 gradients from the recurrence
        dict(name="qk_norm_bwd_train", op="qk_norm_bwd", B=8, S=2048, Hq=32, Hk=32, D=128, R=128, interleaved=False,
             norm="rms", weight=True, fused=True, dtype="bf16", max_pos=2048, grad="f32"),
        # one token of one sequence at 16 heads: the smallest call, where latency counts
        dict(name="gdn_decode_one", op="gdn_decode", B=1, T=1, H=16, Dk=128, Dv=128, slots=1, pool=0, gate=True,
             decay="z", g_min=-5.0, dtype="bf16"),
        # one token of 256 sequences at 32 heads, states taken from a pool by slot
        dict(name="gdn_decode_256", op="gdn_decode", B=256, T=1, H=32, Dk=128, Dv=128, slots=1, pool=16, gate=True,
             decay="z", g_min=-5.0, dtype="bf16"),
        # four drafted tokens of 33 sequences, odd head sizes, exact fp32
        dict(name="gdn_decode_draft", op="gdn_decode", B=33, T=4, H=6, Dk=96, Dv=72, slots=0, pool=0, gate=False,
             decay="log", g_min=-1.0, dtype="f32"),
        # the gradients of a 4096-token prefill at 16 heads
        dict(name="gdn_bwd_prefill_4k", op="gdn_bwd", B=1, S=4096, H=16, Dk=128, Dv=128, decay="z", g_min=-5.0,
             state=True, dtype="bf16"),
        # ragged, slow decay, fp32: sequences that end inside a chunk and head sizes that fill no tile
        dict(name="gdn_bwd_ragged", op="gdn_bwd", B=3, S=777, H=5, Dk=72, Dv=100, decay="log", g_min=-0.25,
             state=True, dtype="f32"),
        # the quantised output of one decode step, 256 sequences at 32 heads
        dict(name="norm_gate_fp8_decode", op="norm_gate_fp8", N=256, H=32, Dv=128, dtype="bf16"),
        # the quantised output of one 8192-token sequence at 32 heads
        dict(name="norm_gate_fp8_8k", op="norm_gate_fp8", N=8192, H=32, Dv=128, dtype="bf16"),
        # the projection of one decode step: 256 rows, weights read once
        dict(name="out_proj_fp8_decode", op="out_proj_fp8", N=256, K=4096, M=4096, out="bf16"),
        # the projection of a whole batch of 8 x 8192 tokens
        dict(name="out_proj_fp8_batch", op="out_proj_fp8", N=65536, K=4096, M=4096, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm", "qk_norm_bwd", "gdn_decode", "gdn_bwd", "norm_gate_fp8", "out_proj_fp8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk_norm", "qk_norm_bwd"):
        D = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
        Hk = rng.randint(1, 32)
        Hq = Hk * rng.choice([1, 1, 2, 4])
        tokens = _log_int(rng, 1, max(1, (1 << 26) // ((Hq + Hk) * D)))
        B = rng.randint(1, min(8, tokens))
        c = dict(op=op, B=B, S=max(1, tokens // B), Hq=Hq, Hk=Hk, D=D, R=rng.choice([0, D // 2, D]),
                 interleaved=rng.random() < 0.5, norm=rng.choice(["l2", "rms"]), weight=rng.random() < 0.6,
                 fused=rng.random() < 0.5, dtype=dtype, max_pos=_log_int(rng, 16, 1 << 20))
        if op == "qk_norm_bwd":
            c["grad"] = rng.choice(["same", "f32"])
        return c
    if op == "gdn_decode":
        Dk = Dv = 128
        if rng.random() < 0.4:
            Dk, Dv = rng.randint(8, 128), rng.randint(8, 128)
        T = rng.choice([1, 1, 1, 2, 3, 4, 5, 8, 13])
        H = rng.randint(1, 32)
        B = _log_int(rng, 1, 8192 // H)
        slots = rng.random() < 0.6
        return dict(op=op, B=B, T=T, H=H, Dk=Dk, Dv=Dv, slots=int(slots), pool=rng.randint(0, 9) if slots else 0,
                    gate=rng.random() < 0.5, decay=rng.choice(["z", "log"]), g_min=rng.choice([-0.1, -1.0, -5.0, -20.0]),
                    dtype=dtype)
    if op == "gdn_bwd":
        Dk = Dv = 128
        if rng.random() < 0.4:
            Dk, Dv = rng.randint(16, 128), rng.randint(16, 128)
        H = rng.randint(1, 16)
        S = _log_int(rng, 1, 4096)
        B = rng.randint(1, max(1, min(6, 65536 // (S * H))))
        return dict(op=op, B=B, S=S, H=H, Dk=Dk, Dv=Dv, decay=rng.choice(["z", "log"]),
                    g_min=rng.choice([-0.25, -1.0, -5.0, -20.0]), state=rng.random() < 0.6, dtype=dtype)
    if op == "norm_gate_fp8":
        Dv = rng.choice([32, 48, 64, 80, 96, 128, 128, 128])
        H = rng.randint(1, 48)
        return dict(op=op, N=_log_int(rng, 1, (1 << 25) // (H * Dv)), H=H, Dv=Dv, dtype=dtype)
    K = 16 * rng.randint(4, 512) if rng.random() < 0.5 else rng.choice([1024, 2048, 4096])
    M = rng.randint(64, 8192) if rng.random() < 0.3 else 128 * rng.randint(1, 64)
    return dict(op=op, N=_log_int(rng, 1, min(65536, (1 << 39) // (K * M))), K=K, M=M, out=rng.choice(["bf16", "bf16", "f32"]))


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def unit(*shape, dtype):  # queries and keys as the recurrence takes them: unit vectors
        x = torch.randn(shape, generator=g, device="cuda")
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    c, op = case, case["op"]
    s = {"case": c}
    if op in ("qk_norm", "qk_norm_bwd"):
        dt = DTYPES[c["dtype"]]
        B, S, Hq, Hk, D = (c[n] for n in ("B", "S", "Hq", "Hk", "D"))
        if c["fused"]:  # views of the rows of one projection: queries, keys, then values of as many heads as the keys
            rows = normal(B, S, (Hq + 2 * Hk) * D, dtype=dt)
            s["q"] = rows[..., :Hq * D].unflatten(-1, (Hq, D))
            s["k"] = rows[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        else:
            s["q"], s["k"] = normal(B, S, Hq, D, dtype=dt), normal(B, S, Hk, D, dtype=dt)
        s["qw"] = 1.0 + normal(D, std=0.1) if c["weight"] else None
        s["kw"] = 1.0 + normal(D, std=0.1) if c["weight"] else None
        s["pos"] = s["inv"] = None
        if c["R"]:
            s["inv"] = (10000.0 ** (-torch.arange(0, c["R"], 2, device="cuda", dtype=torch.float64) / c["R"])).float()
            first = torch.randint(0, c["max_pos"], (B, 1), generator=g, device="cuda")
            s["pos"] = first + torch.arange(S, device="cuda")
        if op == "qk_norm_bwd":
            gt = torch.float32 if c["grad"] == "f32" else dt
            s["dyq"], s["dyk"] = normal(B, S, Hq, D, dtype=gt), normal(B, S, Hk, D, dtype=gt)
    elif op == "gdn_decode":
        dt = DTYPES[c["dtype"]]
        B, T, H, Dk, Dv = (c[n] for n in ("B", "T", "H", "Dk", "Dv"))
        s["q"], s["k"] = unit(B, T, H, Dk, dtype=dt), unit(B, T, H, Dk, dtype=dt)
        s["v"] = normal(B, T, H, Dv, dtype=dt)
        s["beta"] = torch.rand((B, T, H), generator=g, device="cuda").to(dt)
        z = normal(B, T, H)
        s["z"], s["log"] = (z.to(dt), None) if c["decay"] == "z" else (None, c["g_min"] * torch.sigmoid(z))
        s["gate"] = normal(B, T, H, Dv, dtype=dt) if c["gate"] else None
        n = B + c["pool"]
        s["state"] = normal(n, H, Dk, Dv, std=0.02)
        s["slots"] = torch.randperm(n, generator=g, device="cuda")[:B].int() if c["slots"] else None
    elif op == "gdn_bwd":
        dt = DTYPES[c["dtype"]]
        B, S, H, Dk, Dv = (c[n] for n in ("B", "S", "H", "Dk", "Dv"))
        s["q"], s["k"] = unit(B, S, H, Dk, dtype=dt), unit(B, S, H, Dk, dtype=dt)
        s["v"] = normal(B, S, H, Dv, dtype=dt)
        s["beta"] = torch.rand((B, S, H), generator=g, device="cuda").to(dt)
        z = normal(B, S, H)
        s["z"], s["log"] = (z.to(dt), None) if c["decay"] == "z" else (None, c["g_min"] * torch.sigmoid(z))
        s["do"] = normal(B, S, H, Dv, dtype=dt)
        s["s0"] = normal(B, H, Dk, Dv, std=0.02) if c["state"] else None
        s["dsT"] = normal(B, H, Dk, Dv, std=0.1) if c["state"] else None
    elif op == "norm_gate_fp8":
        dt = DTYPES[c["dtype"]]
        s["o"], s["gate"] = (normal(c["N"], c["H"], c["Dv"], dtype=dt, std=sd) for sd in (0.1, 1.0))
    else:
        N, K, M = c["N"], c["K"], c["M"]
        x = normal(N, K, dtype=torch.bfloat16) * normal(N, 1).abs().to(torch.bfloat16)
        s["x"], s["xs"] = _quant(x.float(), 1)
        s["w"], s["ws"] = _quant(normal(M, K, std=K ** -0.5), 128)
        s["out"] = DTYPES[c["out"]]
    return s


# ---------------------------------------------------------------- plain forms
def _pad(x, dim, to):
    """`x` with zeros behind it along `dim`, up to a multiple of `to`."""
    n = -x.shape[dim] % to
    if not n:
        return x
    shape = list(x.shape)
    shape[dim] = n
    return torch.cat([x, x.new_zeros(shape)], dim)


def _blocks(x, rows):
    """A (N, K) matrix as (N / rows, rows, K / 128, 128) blocks, zeros behind its edges."""
    x = _pad(_pad(x, 0, rows), 1, 128)
    return x.view(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def _quant(x, rows):
    """e4m3 values and the fp32 scale of each (rows x 128) block: the block's largest magnitude over 448."""
    b = _blocks(x, rows)
    amax = b.abs().amax(dim=(1, 3))
    scale = torch.where(amax > 0, (amax / E4M3_MAX).clamp_min(TINY), torch.ones_like(amax))
    v = (b / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    v = v.reshape(b.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]].contiguous()
    return v.to(torch.float8_e4m3fn), scale


def _dequant(x, scale, rows, dtype):
    b = _blocks(x.to(dtype), rows) * scale.to(dtype)[:, None, :, None]
    return b.reshape(b.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]]


def _angles(s, dtype):
    """cos and sin of position times frequency, (B, S, 1, R / 2); the angle in 64 bits whatever the result's type."""
    a = s["pos"].double()[..., None, None] * s["inv"].double()
    return a.cos().to(dtype), a.sin().to(dtype)


def _rotate(x, R, interleaved, cos, sin):
    """The first R channels of `x` turned in pairs: (i, i + R/2), or (2i, 2i + 1) where interleaved."""
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _inv_norm(x, norm, eps):
    n = x.square().sum(-1, keepdim=True)
    return (n + eps).rsqrt() if norm == "l2" else (n / x.shape[-1] + eps).rsqrt()


EPS = 1e-6


def _plain_qk_norm(s):
    c = s["case"]
    cs = _angles(s, torch.float32) if c["R"] else None

    def one(x, w):
        y = x.float()
        y = y * _inv_norm(y, c["norm"], EPS)
        y = y if w is None else y * w
        return (y if cs is None else _rotate(y, c["R"], c["interleaved"], *cs)).to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_qk_norm_bwd(s):
    c = s["case"]
    cs = _angles(s, torch.float32) if c["R"] else None
    share = 1.0 if c["norm"] == "l2" else 1.0 / c["D"]

    def one(x, w, dy):
        x, dt = x.float(), x.dtype
        g = dy.float()
        if cs is not None:  # the rotation back
            g = _rotate(g, c["R"], c["interleaved"], cs[0], -cs[1])
        r = _inv_norm(x, c["norm"], EPS)
        dw = None if w is None else (g * x * r).double().sum((0, 1, 2)).float()
        g = g if w is None else g * w
        dx = r * (g - x * ((g * x).sum(-1, keepdim=True) * r * r * share))
        return dx.to(dt), dw

    dq, dqw = one(s["q"], s["qw"], s["dyq"])
    dk, dkw = one(s["k"], s["kw"], s["dyk"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _norm_gate(o, gate, eps):
    return o * (o.square().mean(-1, keepdim=True) + eps).rsqrt() * torch.sigmoid(gate)


def _plain_gdn_decode(s):
    c = s["case"]
    dt = s["q"].dtype
    q, k, v, beta = (s[n].float() for n in ("q", "k", "v", "beta"))
    alpha = (s["log"] if s["z"] is None else c["g_min"] * torch.sigmoid(s["z"].float())).exp()
    at = slice(None) if s["slots"] is None else s["slots"].long()
    S, out = s["state"][at], []
    for t in range(c["T"]):  # each token reads the state that the one before it left
        S = alpha[:, t, :, None, None] * S
        r = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(-2))
        S = S + k[:, t, :, :, None] * r[..., None, :]
        out.append((q[:, t, :, :, None] * S).sum(-2))
    s["state"][at] = S
    o = torch.stack(out, 1)
    if s["gate"] is not None:
        o = _norm_gate(o, s["gate"].float(), EPS)
    return {"o": o.to(dt), "state": s["state"]}


def _plain_gdn_bwd(s):
    """The chunk form, 64 tokens a chunk: everything inside a chunk as matrix products over all chunks at once; only the
    state forwards and its gradient backwards go from chunk to chunk."""
    c, C = s["case"], 64
    B, S, H = c["B"], c["S"], c["H"]
    n = -(-S // C)

    def chunked(x):  # (B, S, H, ...) -> (B, H, n, C, ...)
        x = _pad(x, 1, C)
        return x.view(B, n, C, *x.shape[2:]).movedim(3, 1)

    q, k, v, do, beta = (chunked(s[m].float()) for m in ("q", "k", "v", "do", "beta"))
    raw = s["log"] if s["z"] is None else s["z"].float()
    g = chunked(raw if s["z"] is None else c["g_min"] * torch.sigmoid(raw))
    G = g.double().cumsum(-1)  # differences of far sums: 64 bits
    low = torch.ones(C, C, device=q.device).tril()
    E = torch.exp((G[..., :, None] - G[..., None, :]) * low).float() * low
    eG, eD = G.exp().float()[..., None], (G[..., -1:] - G).exp().float()[..., None]
    gamma = G[..., -1].exp().float()[..., None, None]
    b = beta[..., None]
    A = b * (k @ k.mT) * E * low.tril(-1)
    M = (q @ k.mT) * E
    # T = (I + A)^-1: A is strictly lower, so its 64th power is zero and six factors are the whole series
    P = -A.double()
    T = torch.eye(C, device=q.device, dtype=torch.float64) + P
    P = P @ P; T = T + T @ P
    P = P @ P; T = T + T @ P
    P = P @ P; T = T + T @ P
    P = P @ P; T = T + T @ P
    P = P @ P; T = T + T @ P
    T = T.float()
    Bk, Bv = b * k * eG, b * v
    W, U, Qg, Kd = T @ Bk, T @ Bv, q * eG, k * eD
    St = s["s0"] if s["s0"] is not None else torch.zeros(B, H, c["Dk"], c["Dv"], device=q.device)
    Ss, Vs = [], []
    for i in range(n):  # the state enters each chunk as the one before it left it
        Ss.append(St)
        Vs.append(U[:, :, i] - W[:, :, i] @ St)
        St = gamma[:, :, i] * St + Kd[:, :, i].mT @ Vs[-1]
    Sn, V = torch.stack(Ss, 2), torch.stack(Vs, 2)
    dS = s["dsT"] if s["dsT"] is not None else torch.zeros_like(St)
    dSs, dVs = [], []
    for i in reversed(range(n)):
        dSs.append(dS)
        dVs.append(M[:, :, i].mT @ do[:, :, i] + Kd[:, :, i] @ dS)
        dS = gamma[:, :, i] * dS + Qg[:, :, i].mT @ do[:, :, i] - W[:, :, i].mT @ dVs[-1]
    dSn, dV = torch.stack(dSs[::-1], 2), torch.stack(dVs[::-1], 2)
    dQg, dKd = do @ Sn.mT, V @ dSn.mT
    dM = (do @ V.mT) * low
    dW = -dV @ Sn.mT
    dT = dV @ Bv.mT + dW @ Bk.mT
    dBv, dBk = T.mT @ dV, T.mT @ dW
    dA = -(T.mT @ dT @ T.mT) * low.tril(-1)
    dP = b * dA * E  # through the products of keys with keys
    dMe = dM * E
    dq = dQg * eG + dMe @ k
    dk = b * eG * dBk + eD * dKd + dP @ k + dP.mT @ k + dMe.mT @ q
    dbeta = (dBv * v).sum(-1) + (dBk * k * eG).sum(-1) + (dA * (k @ k.mT) * E).sum(-1)
    # log decay t is in every pair (r, i) with i < t <= r: sums over those pairs, with nothing to cancel
    X = dA * A + dM * M * low.tril(-1)
    below = (X.cumsum(-1) - X) * low  # [r, t]: the sum over i < t, for t <= r
    late = (dQg * Qg).sum(-1) + (dBk * Bk).sum(-1)
    early = (dKd * Kd).sum(-1)
    dg = below.sum(-2) + late.flip(-1).cumsum(-1).flip(-1) + early.cumsum(-1) - early
    dg = dg + (dSn * Sn).sum((-2, -1))[..., None] * gamma[..., 0]

    def flat(x):
        return x.movedim(1, 3).flatten(1, 2)[:, :S].contiguous()

    dg = flat(dg)
    if s["z"] is None:
        dz = torch.where((raw >= c["g_min"]) & (raw <= 0), dg, torch.zeros_like(dg))
    else:
        sg = torch.sigmoid(raw)
        dz = dg * c["g_min"] * sg * (1 - sg)
    return {"dq": flat(dq), "dk": flat(dk), "dv": flat(b * dBv), "dbeta": flat(dbeta), "dz": dz, "ds0": dS}


def _plain_norm_gate_fp8(s):
    x = _norm_gate(s["o"].float(), s["gate"].float(), EPS)
    v, scale = _quant(x.flatten(1), 1)
    return {"x": v, "scale": scale}


def _plain_out_proj_fp8(s):
    x = _dequant(s["x"], s["xs"], 1, torch.float32)
    w = _dequant(s["w"], s["ws"], 128, torch.float32)
    return (x @ w.mT).to(s["out"])


PLAIN = {"qk_norm": _plain_qk_norm, "qk_norm_bwd": _plain_qk_norm_bwd, "gdn_decode": _plain_gdn_decode,
         "gdn_bwd": _plain_gdn_bwd, "norm_gate_fp8": _plain_norm_gate_fp8, "out_proj_fp8": _plain_out_proj_fp8}


# ---------------------------------------------------------------- the framework's entry points
def _own(s):
    import kimi_delta_attention_21_b200 as K
    c, op = s["case"], s["case"]["op"]
    if op in ("qk_norm", "qk_norm_bwd"):
        kw = dict(norm=c["norm"], eps=EPS, q_weight=s["qw"], k_weight=s["kw"], positions=s["pos"], inv_freq=s["inv"],
                  interleaved=c["interleaved"])
        if op == "qk_norm":
            return K.qk_norm(s["q"], s["k"], **kw)
        return K.qk_norm_bwd(s["q"], s["k"], s["dyq"], s["dyk"], **kw)
    if op == "gdn_decode":
        o = K.gdn_decode_step(s["q"], s["k"], s["v"], s["beta"], s["state"], z=s["z"], log_decay=s["log"],
                              g_min=c["g_min"], gate_logits=s["gate"], eps=EPS, slots=s["slots"])
        return {"o": o, "state": s["state"]}
    if op == "gdn_bwd":
        r = K.gdn_chunk_bwd(s["q"], s["k"], s["v"], s["beta"], s["do"], z=s["z"], log_decay=s["log"], g_min=c["g_min"],
                            initial_state=s["s0"], d_final_state=s["dsT"])
        return {"dq": r["dq"], "dk": r["dk"], "dv": r["dv"], "dbeta": r["dbeta"],
                "dz": r["dlog_decay" if s["z"] is None else "dz"], "ds0": r["d_initial_state"]}
    if op == "norm_gate_fp8":
        x, scale = K.norm_gate_fp8(s["o"], s["gate"], eps=EPS)
        return {"x": x, "scale": scale}
    return K.out_proj_fp8(s["x"], s["xs"], s["w"], s["ws"], out_dtype=s["out"])


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    es = 2 if c.get("dtype") == "bf16" else 4
    if op in ("qk_norm", "qk_norm_bwd"):
        rows = c["B"] * c["S"]
        n = rows * (c["Hq"] + c["Hk"]) * c["D"]
        pos = rows * 8 + 2 * c["R"] if c["R"] else 0
        if op == "qk_norm":
            return {"bytes": 2 * n * es + pos, "flops": n * (4 + (3 if c["R"] else 0))}
        gs = 4 if c["grad"] == "f32" else es
        return {"bytes": n * (2 * es + gs) + pos, "flops": n * (10 + (3 if c["R"] else 0))}
    if op == "gdn_decode":
        n, bh = c["B"] * c["T"] * c["H"], c["B"] * c["H"]
        vec = n * ((2 * c["Dk"] + c["Dv"] * (3 if c["gate"] else 2) + 1) * es + (es if c["decay"] == "z" else 4))
        return {"bytes": bh * 8 * c["Dk"] * c["Dv"] + vec + (4 * c["B"] if c["slots"] else 0),
                "flops": n * 7 * c["Dk"] * c["Dv"]}
    if op == "gdn_bwd":
        n, C, Dk, Dv = c["B"] * c["S"] * c["H"], min(64, c["S"]), c["Dk"], c["Dv"]
        states = c["B"] * c["H"] * Dk * Dv * 4 * (3 if c["state"] else 1)
        bts = n * ((2 * Dk + 2 * Dv + 1) * es + (es if c["decay"] == "z" else 4) + (2 * Dk + Dv + 2) * 4) + states
        # per token, in products of a chunk: 6 with the state or its gradient forwards and back, 3 in the gradients; the
        # triangles between the chunk's tokens: K K, Q K, W, dM, dW K, T'dW, and K, Q with dM, dA (5) over D_k; U, M'dO,
        # dO V, dV V, T'dV over D_v
        per = 2 * Dk * Dv * 9 + C * (11 * Dk + 5 * Dv)
        return {"bytes": bts, "flops": n * per}
    if op == "norm_gate_fp8":
        n, K = c["N"] * c["H"] * c["Dv"], c["H"] * c["Dv"]
        return {"bytes": n * (2 * es + 1) + c["N"] * -(-K // 128) * 4, "flops": n * 8}
    N, K, M = c["N"], c["K"], c["M"]
    kb = -(-K // 128)
    return {"bytes": N * K + M * K + 4 * kb * (N + -(-M // 128)) + N * M * (2 if c["out"] == "bf16" else 4),
            "flops": 2 * N * K * M}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm": _exact_norm, "qk_norm_bwd": _exact_norm_bwd, "gdn_decode": _exact_decode, "gdn_bwd": _exact_bwd,
            "norm_gate_fp8": _exact_norm_gate, "out_proj_fp8": _exact_proj}[case["op"]](s, case)


def _turn(x, c, s, back=False):
    """Rotation as a product of complex numbers."""
    R = c["R"]
    if not R:
        return x
    ang = torch.einsum("bs,f->bsf", s["pos"].double(), s["inv"].double())[:, :, None, :]
    phase = torch.polar(torch.ones_like(ang), -ang if back else ang)
    h = x[..., :R]
    if c["interleaved"]:
        pairs = torch.view_as_complex(h.reshape(*h.shape[:-1], R // 2, 2).contiguous()) * phase
        h = torch.view_as_real(pairs).reshape(h.shape)
    else:
        pairs = torch.complex(h[..., :R // 2].contiguous(), h[..., R // 2:].contiguous()) * phase
        h = torch.cat([pairs.real, pairs.imag], -1)
    return torch.cat([h, x[..., R:]], -1)


def _exact_norm(s, c):
    def one(x, w):
        x = x.double()
        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        y = x / torch.sqrt((size if c["norm"] == "l2" else size / c["D"]) + EPS)
        return _turn(y if w is None else y * w.double(), c, s)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _exact_norm_bwd(s, c):
    def one(x, w, dy):
        x = x.double()
        up = _turn(dy.double(), c, s, back=True)
        div = 1 if c["norm"] == "l2" else c["D"]
        size = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / div + EPS).sqrt()
        y = x / size
        dw = None if w is None else torch.einsum("bshd,bshd->d", up, y)
        up = up if w is None else up * w.double()
        return (up - y * torch.einsum("bshd,bshd->bsh", up, y)[..., None] / div) / size, dw

    (dq, dqw), (dk, dkw) = one(s["q"], s["qw"], s["dyq"]), one(s["k"], s["kw"], s["dyk"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _decays(s, c):
    return torch.exp(s["log"].double() if s["z"] is None else c["g_min"] / (1 + torch.exp(-s["z"].double())))


def _exact_decode(s, c):
    a = _decays(s, c)
    rows = torch.arange(c["B"], device="cuda") if s["slots"] is None else s["slots"].long()
    state = s["state"].double()
    S, out = state[rows], []
    for t in range(c["T"]):
        q, k, v = (s[m][:, t].double() for m in ("q", "k", "v"))
        S = a[:, t, :, None, None] * S
        wrong = v - torch.einsum("bhkv,bhk->bhv", S, k)
        S = S + torch.einsum("bhk,bhv->bhkv", k, s["beta"][:, t].double()[..., None] * wrong)
        out.append(torch.einsum("bhkv,bhk->bhv", S, q))
    state[rows] = S
    o = torch.stack(out, 1)
    if s["gate"] is not None:
        o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) / (1 + torch.exp(-s["gate"].double()))
    return {"o": o, "state": state}


def _exact_bwd(s, c):
    """Token by token: every state kept on the way forward, each line of a step differentiated on the way back."""
    B, S, H, Dk, Dv = (c[m] for m in ("B", "S", "H", "Dk", "Dv"))
    if S * B * H * Dk * Dv > 1 << 31:
        return None
    a = _decays(s, c)
    q, k, v, beta, do = (s[m].double().transpose(0, 1).flatten(1, 2) for m in ("q", "k", "v", "beta", "do"))
    a = a.transpose(0, 1).flatten(1, 2)
    St = s["s0"].double().flatten(0, 1) if s["s0"] is not None else q.new_zeros(B * H, Dk, Dv)
    before = q.new_empty(S, B * H, Dk, Dv)
    for t in range(S):
        before[t] = St
        D = a[t, :, None, None] * St
        r = beta[t, :, None] * (v[t] - torch.bmm(k[t, :, None], D)[:, 0])
        St = torch.baddbmm(D, k[t, :, :, None], r[:, None])
    dS = s["dsT"].double().flatten(0, 1) if s["dsT"] is not None else torch.zeros_like(St)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    db, da = torch.empty_like(beta), torch.empty_like(a)
    for t in reversed(range(S)):
        D = a[t, :, None, None] * before[t]
        e = v[t] - torch.bmm(k[t, :, None], D)[:, 0]
        r = beta[t, :, None] * e
        now = torch.baddbmm(D, k[t, :, :, None], r[:, None])
        dq[t] = torch.bmm(now, do[t, :, :, None])[..., 0]
        dS = torch.baddbmm(dS, q[t, :, :, None], do[t, :, None])
        dr = torch.bmm(k[t, :, None], dS)[:, 0]
        db[t] = (dr * e).sum(-1)
        dv[t] = beta[t, :, None] * dr
        dk[t] = torch.bmm(dS, r[..., None])[..., 0] - torch.bmm(D, dv[t, :, :, None])[..., 0]
        dS = torch.baddbmm(dS, k[t, :, :, None], dv[t, :, None], alpha=-1)
        da[t] = (dS * D).sum((-2, -1))  # times the decay: the gradient of its logarithm
        dS = a[t, :, None, None] * dS

    def back(x):
        return x.unflatten(1, (B, H)).transpose(0, 1)

    da = back(da)
    if s["z"] is None:
        dz = da * ((s["log"] >= c["g_min"]) & (s["log"] <= 0))
    else:
        p = 1 / (1 + torch.exp(-s["z"].double()))
        dz = da * c["g_min"] * p * (1 - p)
    return {"dq": back(dq), "dk": back(dk), "dv": back(dv), "dbeta": back(db), "dz": dz, "ds0": dS.unflatten(0, (B, H))}


def _exact_norm_gate(s, c):
    o = s["o"].double()
    x = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) / (1 + torch.exp(-s["gate"].double()))
    x = torch.nn.functional.pad(x.flatten(1), (0, -(c["H"] * c["Dv"]) % 128))
    scale = x.unflatten(1, (-1, 128)).abs().amax(-1) / E4M3_MAX
    return {"x": None, "scale": torch.where(scale > 0, scale, torch.ones_like(scale))}


def _exact_proj(s, c):
    xs = s["xs"].double().repeat_interleave(128, 1)[:, :c["K"]]
    ws = s["ws"].double().repeat_interleave(128, 0)[:c["M"]].repeat_interleave(128, 1)[:, :c["K"]]
    return (s["x"].double() * xs) @ (s["w"].double() * ws).mT

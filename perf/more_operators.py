"""Cases and plain forms of two more operators of the layers around the scan:
the gated delta rule (the other update of a matrix state, chunked for prompts
and recurrent for single tokens and drafts) and the norms before and after a
block with its gate, its residual scale and the residual stream between them.

``run`` computes an operator in plain torch where ``own`` is false and calls
the library's entry point where it is true; ``exact`` is the definition in 64
bits, written apart from both.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5          # of the norms
EPS_QK = 1e-6       # of the keys' and queries' own norms
CHUNK = 64          # of the plain form


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of 64 sequences through a layer of the Llama-hybrid's size: the states' traffic.
        dict(name="delta_step", op="delta", batch=64, tokens=1, heads=32, headdim=128, dkey=128, groups=8, dtype="bf16",
             l2=True, init=True, idx=False, pad=0),
        # One token of one sequence: latency.
        dict(name="delta_step_one", op="delta", batch=1, tokens=1, heads=32, headdim=128, dkey=128, groups=8,
             dtype="bf16", l2=True, init=True, idx=False, pad=0),
        # The verify step: the last token and eight drafts of 64 sequences, with the state after the accepted index.
        dict(name="delta_verify", op="delta", batch=64, tokens=9, heads=32, headdim=128, dkey=128, groups=8,
             dtype="bf16", l2=True, init=True, idx=True, pad=0),
        # A batch of prompts of the 2.7B layer's length through the same layer.
        dict(name="delta_prompt", op="delta", batch=8, tokens=2048, heads=32, headdim=128, dkey=128, groups=8,
             dtype="bf16", l2=True, init=False, idx=False, pad=0),
        # One long document: few heads, so the chain of chunks sets the time.
        dict(name="delta_long", op="delta", batch=1, tokens=16384, heads=32, headdim=128, dkey=128, groups=8,
             dtype="bf16", l2=True, init=False, idx=False, pad=0),
        # A short continuation of two sequences through a narrow layer, from slices of a projection's rows.
        dict(name="delta_short", op="delta", batch=2, tokens=300, heads=16, headdim=64, dkey=64, groups=16,
             dtype="bf16", l2=True, init=True, idx=True, pad=24),
        # fp32, ragged length, head sizes that are no power of two, keys normalised by the caller, no batch of 2^n.
        dict(name="delta_odd", op="delta", batch=3, tokens=1021, heads=10, headdim=80, dkey=96, groups=5, dtype="f32",
             l2=False, init=True, idx=True, pad=3),
        # Between two blocks of one decode step at the Llama-hybrid's width: latency.
        dict(name="norms_step", op="norms", batch=64, tokens=1, dim=4096, dtype="bf16", stream="bf16", post=True,
             gate="token", act="sigmoid", layer_scale=False, pad=32),
        # Between two blocks of a prompt at the 2.7B layer's width: residual stream in fp32, no gate.
        dict(name="norms_prompt", op="norms", batch=8, tokens=2048, dim=5120, dtype="bf16", stream="f32", post=False,
             gate="none", act="none", layer_scale=False, pad=0),
        # The same width with everything: norm after the block, a gate for each token, scale for each channel.
        dict(name="norms_gated", op="norms", batch=8, tokens=2048, dim=4096, dtype="bf16", stream="bf16", post=True,
             gate="token", act="silu", layer_scale=True, pad=64),
        # fp32 with an odd width and a gate for each sequence, rows that start at no 16-byte boundary.
        dict(name="norms_odd", op="norms", batch=3, tokens=1021, dim=2049, dtype="f32", stream="f32", post=True,
             gate="sequence", act="none", layer_scale=True, pad=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.65:
        tokens = rng.choice([1, rng.randint(2, 16), _log(rng, 17, 4096), _log(rng, 17, 4096)])
        dkey = rng.choice([32, 48, 64, 96, 128, 128, 192, 256])
        headdim = rng.choice([16, 32, 64, 80, 128, 128, 256])
        groups = rng.choice([1, 2, 3, 4, 8])
        heads = groups * rng.randint(1, max(1, 32 // groups))
        most = max(1, 4_000_000_000 // (tokens * heads * headdim * dkey * (2 if dtype == "f32" else 1)))
        states = max(1, 60_000_000 // (heads * headdim * dkey))
        return dict(op="delta", batch=min(most, states, _log(rng, 1, 128)), tokens=tokens, heads=heads,
                    headdim=headdim, dkey=dkey, groups=groups, dtype=dtype, l2=rng.random() < 0.6,
                    init=rng.random() < 0.5, idx=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 24, 5]))
    dim = 8 * _log(rng, 8, 1000) + rng.choice([0, 0, 0, 1, 2, 4])
    tokens = rng.choice([1, _log(rng, 2, 4096), _log(rng, 2, 4096)])
    most = max(1, 40_000_000 // (tokens * dim * (2 if dtype == "f32" else 1)))
    return dict(op="norms", batch=min(most, _log(rng, 1, 128)), tokens=tokens, dim=dim, dtype=dtype,
                stream=rng.choice([dtype, "f32"]), post=rng.random() < 0.5,
                gate=rng.choice(["none", "token", "sequence"]), act=rng.choice(["none", "sigmoid", "silu"]),
                layer_scale=rng.random() < 0.5, pad=rng.choice([0, 8, 3, dim]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6151 + 29)
    return g


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _uniform(g, shape, lo=0.0, hi=1.0):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def _rows(values, pad):
    """The values as a slice of longer rows, as a projection leaves them."""
    if pad == 0:
        return values
    b, t, n = values.shape
    rows = values.new_zeros(b, t, n + pad)
    rows[:, :, pad:] = values
    return rows[:, :, pad:]


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    dt = DTYPES[case["dtype"]]
    b, t = case["batch"], case["tokens"]
    if case["op"] == "delta":
        h, p, n, k = case["heads"], case["headdim"], case["dkey"], case["groups"]
        for name in ("q", "k"):
            v = _normal(g, (b, t, k, n))
            if name == "k":                           # keys of neighbouring tokens are alike
                v = v + 0.7 * v.roll(1, 1)
            if not case["l2"]:                        # the caller's own norm
                v = v / v.square().sum(-1, keepdim=True).sqrt()
            s[name] = _rows(v.to(dt).flatten(2), case["pad"]).unflatten(2, (k, n))
        s["v"] = _rows(_normal(g, (b, t, h * p), dt), case["pad"]).unflatten(2, (h, p))
        step = torch.exp(_uniform(g, (h,), math.log(1e-3), math.log(1e-1)))
        rate = torch.exp(_uniform(g, (h,), 0.0, math.log(16.0)))
        raw = _normal(g, (b, t, h)) + torch.log(torch.expm1(step))
        s["g"] = -rate * (torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())))
        s["beta"] = 1.0 / (1.0 + torch.exp(-_normal(g, (b, t, h))))
        s["init"] = _normal(g, (b, h, p, n), scale=0.1) if case["init"] else None
        s["idx"] = torch.randint(0, t, (b,), generator=g, device="cuda", dtype=torch.int32) if case["idx"] else None
        return s
    d = case["dim"]
    s["x"] = _rows(_normal(g, (b, t, d), dt, 0.5), case["pad"])
    s["residual"] = _normal(g, (b, t, d), DTYPES[case["stream"]], 2.0)
    s["gate"] = None if case["gate"] == "none" else _rows(
        _normal(g, (b, 1 if case["gate"] == "sequence" else t, d), dt), case["pad"]).expand(b, t, d)
    s["post_weight"] = 1.0 + _normal(g, (d,), scale=0.1) if case["post"] else None
    s["layer_scale"] = _uniform(g, (d,), 0.1, 1.0) if case["layer_scale"] else None
    s["weight"] = 1.0 + _normal(g, (d,), scale=0.1)
    s["scales"] = (1.0, 0.7)                          # of the residual stream and of the block
    return s


# -------------------------------------------------------------- plain forms
def _delta_inputs32(s):
    c = s["case"]
    q, k, v = (s[name].float().movedim(2, 1) for name in ("q", "k", "v"))       # [b, heads, t, dim]
    if c["l2"]:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + EPS_QK)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + EPS_QK)
    q = q * c["dkey"] ** -0.5
    each = c["heads"] // c["groups"]
    return q.repeat_interleave(each, 1), k.repeat_interleave(each, 1), v, s["g"].movedim(2, 1), s["beta"].movedim(2, 1)


def _delta_tokens(s):
    """Token by token: a few tokens."""
    q, k, v, g, beta = _delta_inputs32(s)
    b, h, t, p = v.shape
    state = v.new_zeros(b, h, p, k.shape[-1]) if s["init"] is None else s["init"]
    at = None if s["idx"] is None else torch.zeros_like(state)
    y = torch.empty_like(v)
    for i in range(t):
        state = state * torch.exp(g[:, :, i, None, None])
        u = beta[:, :, i, None] * (v[:, :, i] - (state * k[:, :, i, None]).sum(-1))
        state = state + u[..., None] * k[:, :, i, None]
        y[:, :, i] = (state * q[:, :, i, None]).sum(-1)
        if at is not None:
            at = torch.where((s["idx"] == i)[:, None, None, None], state, at)
    return y, state, at


def _delta_chunks(s):
    """Chunk by chunk with matrix products: prompts."""
    q, k, v, g, beta = _delta_inputs32(s)
    b, h, t, p = v.shape
    n, c = k.shape[-1], CHUNK
    nc = -(-t // c)

    def cut(x):                                       # [b, h, nc, c, ...], zeros past the end
        full = x.new_zeros(b, h, nc * c, *x.shape[3:])
        full[:, :, :t] = x
        return full.unflatten(2, (nc, c))

    q, k, v, g, beta = cut(q), cut(k), cut(v), cut(g), cut(beta)
    total = g.double().cumsum(3)                      # differences of long sums: 64 bits
    place = torch.arange(c, device=v.device)
    back = total[..., :, None] - total[..., None, :]
    decay = torch.exp(torch.where(place[:, None] >= place, back, torch.zeros_like(back))).float()
    decay = decay * (place[:, None] >= place)
    lower = torch.matmul(k, k.transpose(-1, -2)) * decay * beta[..., None] * (place[:, None] > place)
    solve = torch.zeros_like(lower) + torch.eye(c, device=v.device)
    for i in range(1, c):                             # (1 + lower) solve = 1, row by row, all chunks at once
        solve[..., i, :i] = -(lower[..., i, :i, None] * solve[..., :i, :i]).sum(-2)
    solve = solve * beta[..., None, :]
    within = torch.matmul(q, k.transpose(-1, -2)) * decay
    grown = torch.exp(total).float()[..., None]
    left = torch.exp(total[..., -1:] - total).float()[..., None]
    state = v.new_zeros(b, h, p, n) if s["init"] is None else s["init"]
    at = None if s["idx"] is None else torch.zeros_like(state)
    y = torch.empty_like(v)
    for i in range(nc):
        u = torch.matmul(solve[:, :, i], v[:, :, i] - grown[:, :, i] * torch.matmul(k[:, :, i], state.transpose(-1, -2)))
        y[:, :, i] = grown[:, :, i] * torch.matmul(q[:, :, i], state.transpose(-1, -2)) + torch.matmul(within[:, :, i], u)
        if at is not None:                            # the state after the index, for the sequences it lies here in
            here = (s["idx"].long() - i * c).clamp(0, c - 1)
            share = decay[torch.arange(b, device=v.device), :, i, here][..., None]
            till = grown[torch.arange(b, device=v.device), :, i, here][..., None]
            then = till * state + torch.matmul((share * u).transpose(-1, -2), k[:, :, i])
            at = torch.where((s["idx"].long() // c == i)[:, None, None, None], then, at)
        state = grown[:, :, i, -1, :, None] * state + torch.matmul((left[:, :, i] * u).transpose(-1, -2), k[:, :, i])
    return y.flatten(2, 3)[:, :, :t], state, at


def _delta_plain(s):
    y, state, at = (_delta_tokens if s["case"]["tokens"] <= 16 else _delta_chunks)(s)
    return [y.movedim(1, 2).contiguous().to(s["v"].dtype), state] + ([] if at is None else [at])


def _norms_plain(s):
    c = s["case"]
    x = s["x"].float()
    if c["post"]:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * s["post_weight"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        open_ = 1.0 / (1.0 + torch.exp(-gate))
        x = x * {"none": gate, "sigmoid": open_, "silu": gate * open_}[c["act"]]
    if s["layer_scale"] is not None:
        x = x * s["layer_scale"]
    h = s["scales"][0] * s["residual"].float() + s["scales"][1] * x
    out = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    return [out.to(s["x"].dtype), h.to(s["residual"].dtype)]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"delta": _delta_plain, "norms": _norms_plain}[c["op"]](s)
    import mamba_ssd_scan_06_amd as ssd
    if c["op"] == "delta":
        y, final, at = ssd.ssd_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["init"], s["idx"],
                                               qk_l2norm=c["l2"])
        return [y, final] + ([] if at is None else [at])
    return list(ssd.ssd_residual_norm_fwd(
        s["x"], s["residual"], s["weight"], post_norm=c["post"], post_weight=s["post_weight"], gate=s["gate"],
        gate_activation=None if c["act"] == "none" else c["act"], layer_scale=s["layer_scale"],
        residual_scale=s["scales"][0], branch_scale=s["scales"][1], eps=EPS))


# ------------------------------------------------------------------- costs
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    b, t = case["batch"], case["tokens"]
    if case["op"] == "delta":
        h, p, n, k = case["heads"], case["headdim"], case["dkey"], case["groups"]
        state = 4 * b * h * p * n
        return {"bytes": b * t * (2 * e * (k * n + h * p) + 8 * h) + state * (1 + case["init"] + case["idx"]),
                "flops": 7 * b * t * h * p * n}       # decay, the state's products with key and query, the update
    d = case["dim"]
    r = 2 if case["stream"] == "bf16" else 4
    gates = {"none": 0, "token": t, "sequence": 1}[case["gate"]]
    vectors = 4 * d * (1 + case["post"] + case["layer_scale"])
    return {"bytes": b * d * (t * (2 * e + 2 * r) + gates * e) + vectors,
            "flops": b * t * d * (7 + 4 * case["post"] + (6 if gates else 0) + case["layer_scale"])}


# ------------------------------------------------------- definition, 64 bits
def _exact_delta(s):
    c = s["case"]
    each = c["heads"] // c["groups"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if c["l2"]:
        q = q * torch.rsqrt((q ** 2).sum(3, keepdim=True) + EPS_QK)
        k = k * torch.rsqrt((k ** 2).sum(3, keepdim=True) + EPS_QK)
    b, t, h, p = v.shape
    alpha, beta = torch.exp(s["g"].double()), s["beta"].double()
    m = torch.zeros(b, h, p, c["dkey"], dtype=torch.float64, device=v.device)
    if s["init"] is not None:
        m += s["init"]
    last = None if s["idx"] is None else s["idx"].long()
    at = None if last is None else torch.empty_like(m)
    y = torch.empty_like(v)
    for i in range(t):
        ki = k[:, i].repeat_interleave(each, 1).unsqueeze(3)
        qi = q[:, i].repeat_interleave(each, 1).unsqueeze(3)
        m *= alpha[:, i, :, None, None]
        short = v[:, i].unsqueeze(3) - torch.matmul(m, ki)
        m.addcmul_(short * beta[:, i, :, None, None], ki.transpose(2, 3))
        y[:, i] = torch.matmul(m, qi).squeeze(3) / math.sqrt(c["dkey"])
        if last is not None:
            at[last == i] = m[last == i]
    return [y, m] + ([] if at is None else [at])


def _exact_norms(s):
    c = s["case"]
    d = c["dim"]
    branch = s["x"].double()
    if c["post"]:
        size = torch.linalg.vector_norm(branch, dim=2, keepdim=True)
        branch = branch * torch.rsqrt(size ** 2 / d + EPS) * s["post_weight"].double()
    if s["gate"] is not None:
        gate = s["gate"].double()
        if c["act"] == "sigmoid":
            gate = torch.sigmoid(gate)
        elif c["act"] == "silu":
            gate = gate * torch.sigmoid(gate)
        branch = branch * gate
    if s["layer_scale"] is not None:
        branch = branch * s["layer_scale"].double()
    h = s["residual"].double() * s["scales"][0] + branch * s["scales"][1]
    size = torch.linalg.vector_norm(h, dim=2, keepdim=True)
    return [h * torch.rsqrt(size ** 2 / d + EPS) * s["weight"].double(), h]


def exact(case, seed):
    s = prepare(case, seed)
    return {"delta": _exact_delta, "norms": _exact_norms}[case["op"]](s)

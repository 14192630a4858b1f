"""Cases and plain forms of the operators that stand around the SSD scan: the
short causal convolution before it, the selective scan with one decay per
channel and state index, the gated RMS norm after it, and the verification of
drafted tokens whose accepted index the scans take.

``run`` computes an operator in plain torch where ``own`` is false and calls
the library's entry point where it is true; ``exact`` is the definition in 64
bits, written apart from both.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One decode step of the 2.7B layer's convolution: 64 sequences, x | B | C of one token each.
        dict(name="conv_step", op="conv", batch=64, tokens=1, c0=5120, c1=128, c2=128, pad=5200, width=4, dtype="bf16",
             silu=True, bias=True, init=True, idx=False),
        # The 2.7B layer's prompt: the slice x | B | C of the input projection's rows, split on the way out.
        dict(name="conv_prompt", op="conv", batch=8, tokens=2048, c0=5120, c1=128, c2=128, pad=5200, width=4,
             dtype="bf16", silu=True, bias=True, init=False, idx=True),
        # Odd sizes in fp32: three taps, ragged length, rows that start at no 16-byte boundary.
        dict(name="conv_odd", op="conv", batch=3, tokens=1021, c0=1001, c1=24, c2=40, pad=7, width=3, dtype="f32",
             silu=False, bias=True, init=True, idx=True),
        # One decode step of a selective-scan layer with 5120 channels, 64 sequences.
        dict(name="scan_step", op="scan", batch=64, tokens=1, channels=5120, dstate=16, ngroups=1, dtype="bf16",
             softplus=True, gate=True, init=True, idx=False),
        # A batch of prompts through the same layer.
        dict(name="scan_prompt", op="scan", batch=8, tokens=2048, channels=5120, dstate=16, ngroups=1, dtype="bf16",
             softplus=True, gate=True, init=False, idx=True),
        # One long prompt through a narrow layer: few channels, so the length has to be shared out.
        dict(name="scan_long", op="scan", batch=1, tokens=4093, channels=1536, dstate=16, ngroups=1, dtype="bf16",
             softplus=True, gate=True, init=True, idx=True),
        # fp32 with a wide state, two groups and a channel count that ends inside a tile; steps given, no gate.
        dict(name="scan_wide_state", op="scan", batch=2, tokens=515, channels=1000, dstate=64, ngroups=2, dtype="f32",
             softplus=False, gate=False, init=True, idx=False),
        # Norm of one decode step at the Llama-hybrid layer's width, one norm per B/C group.
        dict(name="norm_step", op="norm", rows=64, dim=4096, ngroups=8, pad=6176, dtype="bf16", gate_first=True),
        # Norm of the 2.7B layer's prompt; z is a slice of the input projection's rows.
        dict(name="norm_prompt", op="norm", rows=16384, dim=5120, ngroups=1, pad=5456, dtype="bf16", gate_first=True),
        # One sequence with eight drafts over a large vocabulary: latency.
        dict(name="verify_one", op="verify", batch=1, drafts=8, vocab=128256, dtype="f32", q=True, ragged=False),
        # A serving batch as in the multi-step verify workload: 64 sequences, eight drafts each.
        dict(name="verify_batch", op="verify", batch=64, drafts=8, vocab=32000, dtype="f32", q=True, ragged=True),
        # Many sequences with drafts from a lookup (no draft distribution) and an odd vocabulary.
        dict(name="verify_lookup", op="verify", batch=256, drafts=4, vocab=50277, dtype="f32", q=False, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        tokens = rng.choice([1, rng.randint(2, 16), _log(rng, 17, 4096)])
        c0 = 8 * _log(rng, 8, 768) + rng.choice([0, 0, 0, 1, 2, 5])
        c1, c2 = rng.choice([(0, 0), (128, 128), (16, 16), (256, 256), (24, 40)])
        most = max(1, 80_000_000 // ((c0 + c1 + c2) * tokens * (2 if dtype == "f32" else 1)))
        return dict(op="conv", batch=min(most, _log(rng, 1, 128)), tokens=tokens, c0=c0, c1=c1, c2=c2,
                    pad=rng.choice([0, 8, 2, 5, c0]), width=rng.choice([2, 3, 4, 4]), dtype=dtype,
                    silu=rng.random() < 0.7, bias=rng.random() < 0.7, init=rng.random() < 0.5, idx=rng.random() < 0.5)
    if op == "scan":
        tokens = rng.choice([1, rng.randint(2, 16), _log(rng, 17, 4093)])
        dstate = rng.choice([8, 16, 16, 32, 64])
        groups = rng.choice([1, 1, 2, 4])
        channels = 8 * groups * _log(rng, 8 // groups, 800 // groups)
        most = max(1, 1_000_000_000 // (channels * tokens * dstate))
        return dict(op="scan", batch=min(most, _log(rng, 1, 64)), tokens=tokens, channels=channels, dstate=dstate,
                    ngroups=groups, dtype=dtype, softplus=rng.random() < 0.7, gate=rng.random() < 0.7,
                    init=rng.random() < 0.5, idx=rng.random() < 0.5)
    if op == "norm":
        groups = rng.choice([1, 1, 2, 8])
        dim = 8 * groups * _log(rng, 8, 1100 // groups) + groups * rng.choice([0, 0, 0, 1, 2])
        rows = min(_log(rng, 1, 16384), 80_000_000 // dim // (2 if dtype == "f32" else 1))
        return dict(op="norm", rows=rows, dim=dim, ngroups=groups, pad=rng.choice([0, 8, 3, dim]), dtype=dtype,
                    gate_first=rng.random() < 0.7)
    vocab = _log(rng, 100, 150000)
    drafts = rng.randint(0, 12)
    most = max(1, 50_000_000 // (vocab * (drafts + 1)))
    return dict(op="verify", batch=min(most, _log(rng, 1, 256)), drafts=drafts, vocab=vocab, dtype=dtype,
                q=rng.random() < 0.7, ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _uniform(g, shape, lo=0.0, hi=1.0):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "conv":
        b, t, w = case["batch"], case["tokens"], case["width"]
        c = case["c0"] + case["c1"] + case["c2"]
        rows = _normal(g, (b, t, c + case["pad"]), dt)
        s["x"] = rows[:, :, case["pad"]:]            # a slice of a projection's rows
        s["weight"] = _normal(g, (c, w), scale=w ** -0.5)
        s["bias"] = _normal(g, (c,), scale=0.1) if case["bias"] else None
        s["init"] = _normal(g, (b, w - 1, c), dt) if case["init"] else None
        s["idx"] = torch.randint(0, t, (b,), generator=g, device="cuda", dtype=torch.int32) if case["idx"] else None
        s["split"] = [k for k in (case["c0"], case["c1"], case["c2"]) if k > 0]
    elif case["op"] == "scan":
        b, t, d, n, k = case["batch"], case["tokens"], case["channels"], case["dstate"], case["ngroups"]
        rank = 8 * ((d + 127) // 128)
        s["u"] = _normal(g, (b, t, d), dt)
        s["z"] = _normal(g, (b, t, 2 * d), dt)[:, :, d:] if case["gate"] else None
        proj = _normal(g, (b, t, rank + 2 * k * n), dt)
        s["B"] = proj[:, :, rank:rank + k * n].unflatten(2, (k, n))
        s["C"] = proj[:, :, rank + k * n:].unflatten(2, (k, n))
        step = torch.exp(_uniform(g, (d,), math.log(1e-3), math.log(1e-1)))
        if case["softplus"]:
            s["delta"] = _normal(g, (b, t, d), dt)
            s["bias"] = torch.log(torch.expm1(step))
        else:
            s["delta"] = (step * torch.exp(_normal(g, (b, t, d), scale=0.5))).to(dt)
            s["bias"] = None
        s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * _uniform(g, (d, n), 0.5, 1.5)
        s["D"] = _normal(g, (d,))
        s["init"] = _normal(g, (b, d, n), scale=0.1) if case["init"] else None
        s["idx"] = torch.randint(0, t, (b,), generator=g, device="cuda", dtype=torch.int32) if case["idx"] else None
    elif case["op"] == "norm":
        r, d = case["rows"], case["dim"]
        s["x"] = _normal(g, (r, d), dt)
        s["z"] = _normal(g, (r, d + case["pad"]), dt)[:, case["pad"]:]
        s["weight"] = 1.0 + _normal(g, (d,), scale=0.1)
    else:
        b, k, v = case["batch"], case["drafts"], case["vocab"]
        logits = _normal(g, (b, k + 1, v), scale=2.0)
        near = logits[:, :k] + _normal(g, (b, k, v), scale=0.7)
        q = torch.softmax(near, dim=-1)
        tok = torch.empty(b, k, device="cuda", dtype=torch.int64)
        for i in range(k):                            # drafts follow the draft distribution
            cut = _uniform(g, (b, 1)).double() * 0.999999
            tok[:, i] = (q[:, i].double().cumsum(1) <= cut).sum(1).clamp(max=v - 1)
        s["p"] = torch.softmax(logits, dim=-1).to(dt)
        s["q"] = q.to(dt) if case["q"] else None
        if not case["q"]:                             # looked-up drafts are often the likeliest token
            top = logits[:, :k].argmax(-1) if k else tok
            tok = torch.where(_uniform(g, (b, k)) < 0.8, top, tok)
        s["tok"] = tok.to(torch.int32)
        s["u"] = _uniform(g, (b, k + 1))
        if not case["q"]:
            s["u"][:, :k] *= 0.2                      # the likeliest of many tokens is still a small share
        s["lens"] = torch.randint(0, k + 1, (b,), generator=g, device="cuda", dtype=torch.int32) \
            if case["ragged"] else None
    return s


# -------------------------------------------------------------- plain forms
def _silu32(v):
    return v / (1.0 + torch.exp(-v))


def _conv_plain(s):
    c, w = s["case"], s["case"]["width"]
    x = s["x"].float()
    b, t, ch = x.shape
    past = torch.zeros(b, w - 1, ch, device=x.device) if s["init"] is None else s["init"].float()
    full = torch.cat([past, x], dim=1)
    acc = torch.zeros_like(x) if s["bias"] is None else s["bias"].expand_as(x).clone()
    for k in range(w):
        acc = acc + s["weight"][:, k] * full[:, k:k + t]
    if c["silu"]:
        acc = _silu32(acc)
    dt = s["x"].dtype
    outs = [o.contiguous().to(dt) for o in acc.split(s["split"], dim=2)]
    final = full[:, t:].to(dt)
    at = None
    if s["idx"] is not None:
        rows = s["idx"].long()[:, None] + 1 + torch.arange(w - 1, device=x.device)
        at = full.gather(1, rows[:, :, None].expand(b, w - 1, ch)).to(dt)
    return outs + [final] + ([] if at is None else [at])


def _softplus32(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _scan_plain(s):
    c = s["case"]
    u, delta = s["u"].float(), s["delta"].float()
    b, t, d = u.shape
    n, k = c["dstate"], c["ngroups"]
    if s["bias"] is not None:
        delta = delta + s["bias"]
    if c["softplus"]:
        delta = _softplus32(delta)
    h = torch.zeros(b, d, n, device=u.device) if s["init"] is None else s["init"].clone()
    at = torch.zeros_like(h) if s["idx"] is not None else None
    du = delta * u
    B, C = s["B"].float(), s["C"].float()
    y = torch.empty_like(u)
    for i in range(t):
        bi = B[:, i].repeat_interleave(d // k, dim=1)
        ci = C[:, i].repeat_interleave(d // k, dim=1)
        h = torch.exp(delta[:, i, :, None] * s["A"]) * h + du[:, i, :, None] * bi
        y[:, i] = (h * ci).sum(-1)
        if at is not None:
            at = torch.where((s["idx"] == i)[:, None, None], h, at)
    y = y + s["D"] * u
    if s["z"] is not None:
        y = y * _silu32(s["z"].float())
    return [y.to(s["u"].dtype), h] + ([] if at is None else [at])


def _norm_plain(s):
    c = s["case"]
    x, gate = s["x"].float(), _silu32(s["z"].float())
    if c["gate_first"]:
        x = x * gate
    parts = x.unflatten(1, (c["ngroups"], -1))
    x = (parts / torch.sqrt((parts * parts).mean(-1, keepdim=True) + 1e-5)).flatten(1) * s["weight"]
    if not c["gate_first"]:
        x = x * gate
    return [x.to(s["x"].dtype)]


def _verify_plain(s):
    p = s["p"]
    b, rows, v = p.shape
    k = rows - 1
    dev = p.device
    lens = torch.full((b,), k, device=dev) if s["lens"] is None else s["lens"].long()
    if k > 0:
        tok = s["tok"].long()
        pt = p[:, :k].gather(2, tok[:, :, None])[:, :, 0].double()
        qt = torch.ones_like(pt) if s["q"] is None else s["q"].gather(2, tok[:, :, None])[:, :, 0].double()
        ok = (s["u"][:, :k].double() * qt < pt) & (torch.arange(k, device=dev) < lens[:, None])
        n = ok.long().cumprod(1).sum(1)
    else:
        tok = torch.zeros(b, 1, device=dev, dtype=torch.long)
        n = torch.zeros(b, device=dev, dtype=torch.long)
    seq = torch.arange(b, device=dev)
    row = p[seq, n].double()
    rejected = n < lens
    if k > 0:
        at = n.clamp(max=k - 1)
        if s["q"] is None:
            less = torch.zeros_like(row)
            less[seq, tok[seq, at]] = row[seq, tok[seq, at]]
        else:
            less = s["q"][seq, at].double()
        rest = (row - less).clamp(min=0)
        rejected = rejected & (rest.sum(1) > 0)       # no mass left by rounding: the target row itself
        row = torch.where(rejected[:, None], rest, row)
    cdf = row.cumsum(1)
    cut = s["u"][:, k].double() * cdf[:, -1]
    nxt = (cdf <= cut[:, None]).sum(1).clamp(max=v - 1)
    place = torch.arange(k + 1, device=dev)
    drafts = torch.cat([s["tok"].long(), torch.zeros(b, 1, device=dev, dtype=torch.long)], dim=1)
    tokens = torch.where(place < n[:, None], drafts, torch.full_like(drafts, -1))
    tokens = torch.where(place == n[:, None], nxt[:, None], tokens)
    return [n.to(torch.int32), nxt.to(torch.int32), tokens.to(torch.int32)]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"conv": _conv_plain, "scan": _scan_plain, "norm": _norm_plain, "verify": _verify_plain}[c["op"]](s)
    import mamba_ssd_scan_06_amd as ssd
    if c["op"] == "conv":
        outs, final, at = ssd.ssd_causal_conv_fwd(s["x"], s["weight"], s["bias"], s["init"], s["idx"],
                                                  split=s["split"], activation="silu" if c["silu"] else None)
        return list(outs) + [final] + ([] if at is None else [at])
    if c["op"] == "scan":
        y, final, at = ssd.ssd_selective_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                                  s["bias"], s["init"], s["idx"], delta_softplus=c["softplus"])
        return [y, final] + ([] if at is None else [at])
    if c["op"] == "norm":
        return [ssd.ssd_gated_norm_fwd(s["x"], s["z"], s["weight"], ngroups=c["ngroups"], eps=1e-5,
                                       norm_before_gate=not c["gate_first"])]
    return list(ssd.ssd_verify_drafts(s["p"], s["tok"], s["u"], s["q"], s["lens"]))


# ------------------------------------------------------------------- costs
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "conv":
        b, t, w = case["batch"], case["tokens"], case["width"]
        c = case["c0"] + case["c1"] + case["c2"]
        state = b * (w - 1) * c * e
        n = 2 * b * t * c * e + 4 * c * (w + bool(case["bias"])) + state * (1 + case["init"] + case["idx"])
        return {"bytes": n, "flops": b * t * c * (2 * w + (4 if case["silu"] else 0))}
    if case["op"] == "scan":
        b, t, d, n, k = case["batch"], case["tokens"], case["channels"], case["dstate"], case["ngroups"]
        state = 4 * b * d * n
        size = e * b * t * (d * (3 + case["gate"]) + 2 * k * n) + 4 * d * (n + 2) \
            + state * (1 + case["init"] + case["idx"])
        return {"bytes": size, "flops": b * t * d * (7 * n + 3 + 6 * case["softplus"] + 5 * case["gate"])}
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        return {"bytes": 3 * n * e + 4 * case["dim"], "flops": 9 * n}
    b, k, v = case["batch"], case["drafts"], case["vocab"]
    rows = 2 if case["q"] and k > 0 else 1
    return {"bytes": b * (v * rows * e + 4 * k + 4 * (k + 1) * 2 + 8), "flops": 3 * b * v * rows}


# ------------------------------------------------------- definition, 64 bits
def _exact_conv(s):
    c = s["case"]
    w = c["width"]
    x = s["x"].double()
    b, t, ch = x.shape
    taps = s["weight"].double()
    held = x.new_zeros(b, w - 1, ch) if s["init"] is None else s["init"].double()
    out = x.new_zeros(b, t, ch)
    for lag in range(w):                              # token t - lag meets tap w - 1 - lag
        if lag < t:
            out[:, lag:] += x[:, :t - lag] * taps[:, w - 1 - lag]
        for i in range(min(lag, t)):                  # the first tokens reach into the held ones
            out[:, i] += held[:, w - 1 + i - lag] * taps[:, w - 1 - lag]
    if s["bias"] is not None:
        out += s["bias"].double()
    if c["silu"]:
        out = out * torch.sigmoid(out)

    def tail(seq, count):                             # the w - 1 inputs before input `count`
        return torch.stack([x[seq, j] if j >= 0 else held[seq, w - 1 + j] for j in range(count - w + 1, count)])

    final = torch.stack([tail(i, t) for i in range(b)])
    res = list(out.split(s["split"], dim=2)) + [final]
    if s["idx"] is not None:
        res.append(torch.stack([tail(i, int(j) + 1) for i, j in enumerate(s["idx"].tolist())]))
    return res


def _exact_scan(s):
    c = s["case"]
    u, delta = s["u"].double(), s["delta"].double()
    b, t, d = u.shape
    n, k = c["dstate"], c["ngroups"]
    if s["bias"] is not None:
        delta = delta + s["bias"].double()
    if c["softplus"]:
        delta = torch.logaddexp(delta, torch.zeros_like(delta))
    du = delta * u
    A = s["A"].double()
    y = s["D"].double() * u
    final = torch.empty(b, d, n, dtype=torch.float64, device=u.device)
    at = torch.empty_like(final)
    last = None if s["idx"] is None else s["idx"].long()
    for m in range(n):                                # each state index by doubling: spans of 1, 2, 4, ... tokens
        coef = torch.exp(delta * A[:, m])
        held = du * s["B"][:, :, :, m].double().repeat_interleave(d // k, dim=2)
        if s["init"] is not None:
            held[:, 0] += coef[:, 0] * s["init"][:, :, m].double()
        span = 1
        while span < t:
            grown = coef[:, span:] * held[:, :-span]
            more = coef[:, span:] * coef[:, :-span]
            held[:, span:] += grown
            coef = torch.cat([coef[:, :span], more], dim=1)
            span *= 2
        y += held * s["C"][:, :, :, m].double().repeat_interleave(d // k, dim=2)
        final[:, :, m] = held[:, -1]
        if last is not None:
            at[:, :, m] = held[torch.arange(b, device=u.device), last]
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    return [y, final] + ([] if last is None else [at])


def _exact_norm(s):
    c = s["case"]
    x, z = s["x"].double(), s["z"].double()
    gate = z * torch.sigmoid(z)
    v = x * gate if c["gate_first"] else x
    out = torch.empty_like(v)
    m = c["dim"] // c["ngroups"]
    for g in range(c["ngroups"]):
        part = v[:, g * m:(g + 1) * m]
        norm = torch.linalg.vector_norm(part, dim=1, keepdim=True)
        out[:, g * m:(g + 1) * m] = part * torch.rsqrt(norm ** 2 / m + 1e-5)
    out *= s["weight"].double()
    return [out if c["gate_first"] else out * gate]


def _exact_verify(s):
    b, rows, v = s["p"].shape
    k = rows - 1
    tok, u = s["tok"].cpu().numpy(), s["u"].cpu().numpy().astype(np.float64)
    lens = np.full(b, k) if s["lens"] is None else s["lens"].cpu().numpy()
    count, nxt = np.zeros(b, np.int32), np.zeros(b, np.int32)
    tokens = np.full((b, k + 1), -1, np.int32)
    for i in range(b):
        p = s["p"][i].float().cpu().numpy().astype(np.float64)
        q = None if s["q"] is None else s["q"][i].float().cpu().numpy().astype(np.float64)
        j = 0
        while j < lens[i] and u[i, j] * (1.0 if q is None else q[j, tok[i, j]]) < p[j, tok[i, j]]:
            j += 1
        rest = p[j].copy()
        if j < lens[i]:
            if q is None:
                rest[tok[i, j]] = 0.0
            else:
                rest = np.maximum(rest - q[j], 0.0)
            rest = rest if rest.any() else p[j]
        total = np.cumsum(rest)
        pick = int(np.searchsorted(total, u[i, k] * total[-1], side="right"))
        count[i], nxt[i] = j, min(pick, v - 1)
        tokens[i, :j], tokens[i, j] = tok[i, :j], nxt[i]
    return [torch.from_numpy(a) for a in (count, nxt, tokens)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm, "verify": _exact_verify}[case["op"]](s)

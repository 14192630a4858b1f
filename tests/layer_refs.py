"""The operators around the scan in fp64 (numpy, from their definitions), each
with a bound on what an fp32 evaluation with one final rounding may differ by.

Bounds are first-order sums of the roundings an fp32 evaluation makes: every
product and sum is off by at most U = 2^-24 of its value, the hardware
exponential and reciprocal by one unit in the last place (2 U), and the final
rounding by half a step of the output's type (2^-8 of the value for bf16, 2^-24
for fp32).  SLACK covers second-order terms; TINY covers results that the
hardware exponential flushes to zero (below 2^-126, times values up to 1e3).
"""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
SLACK = 1.01
TINY = 1e-34


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * v))


def silu(v):
    return v * sigmoid(v)


def silu_rel(v):
    """Relative error of v / (1 + exp(-v)): the exponent -v log2(e) carries two
    roundings (|v| 2 U in e^-v), the exponential 2 U, the sum, reciprocal and
    product U + 2 U + U."""
    return (2.0 * np.abs(v) + 6.0) * U


def rounded(ref, err, dtype):
    """Bound on the stored output: the fp32 error plus the final rounding."""
    return SLACK * (err + HALF_STEP[dtype] * (np.abs(ref) + err)) + TINY


def conv(x, weight, bias, init, idx, act, dtype):
    """(out, bound, final, at): x [b,T,C], weight [C,W]."""
    b, T, C = x.shape
    W = weight.shape[1]
    held = np.zeros((b, W - 1, C)) if init is None else init
    full = np.concatenate([held, x], axis=1)
    acc = np.zeros((b, T, C)) + (0.0 if bias is None else bias)
    mag = np.abs(acc)
    for k in range(W):
        term = weight[:, k] * full[:, k:k + T]
        acc = acc + term
        mag = mag + np.abs(term)
    err = (W + 1) * U * mag
    out = acc
    if act:
        out = silu(acc)
        err = 1.1 * err + silu_rel(acc) * np.abs(out)       # |silu'| <= 1.1
    final = full[:, T:]
    at = None if idx is None else np.stack([full[i, j + 1:j + W] for i, j in enumerate(idx)])
    return out, rounded(out, err, dtype), final, at


def selective_scan(u, delta, A, B, C, D, z, bias, softplus, init, idx, dtype):
    """(y, y_bound, final, final_bound, at, at_bound): B, C [b,T,G,N]."""
    b, T, Dm = u.shape
    N = A.shape[1]
    G = B.shape[2]
    rep = Dm // G
    h = np.zeros((b, Dm, N)) if init is None else init.copy()
    e = np.zeros_like(h)
    at, at_e = (None, None) if idx is None else (np.empty_like(h), np.empty_like(h))

    def keep(t):
        if idx is not None:
            m = idx == t
            at[m], at_e[m] = h[m], e[m]

    keep(-1)
    s = delta + (0.0 if bias is None else bias)
    s_rel = np.full_like(s, U)
    if softplus:
        # The sum delta + bias is off by U |s|, which moves log(1 + e^s) by at
        # most that share of itself; the exponential, reciprocal, series and
        # products add under ten roundings.
        s_rel = (3.0 * np.abs(s) + 10.0) * U
        s = np.logaddexp(s, 0.0)
    y, y_e = np.empty_like(u), np.empty_like(u)
    for t in range(T):
        st = s[:, t, :, None]
        sr = s_rel[:, t, :, None]
        Bt = np.repeat(B[:, t], rep, axis=1)
        Ct = np.repeat(C[:, t], rep, axis=1)
        x = st * A
        a = np.exp(x)
        v = st * u[:, t, :, None] * Bt
        # exp(x): the exponent carries s's error and three roundings.
        a_rel = np.abs(x) * (sr + 3 * U) + 2 * U
        e = a * (e + np.abs(h) * a_rel) + np.abs(v) * (sr + 3 * U)
        h = a * h + v
        e = e + 2 * U * np.abs(h)
        hc = h * Ct
        y[:, t] = hc.sum(-1)
        y_e[:, t] = (np.abs(Ct) * e).sum(-1) + (N + 1) * U * np.abs(hc).sum(-1)
        keep(t)
    if D is not None:
        y_e += 2 * U * np.abs(D * u) + U * np.abs(y + D * u)
        y = y + D * u
    if z is not None:
        g = silu(z)
        y_e = y_e * np.abs(g) + np.abs(y * g) * (silu_rel(z) + U)
        y = y * g
    fin_b = SLACK * e + TINY
    return y, rounded(y, y_e, dtype), h, fin_b, at, None if at is None else SLACK * at_e + TINY


def gated_norm(x, z, weight, groups, eps, norm_first, dtype):
    """(out, bound): x [rows,dim]."""
    rows, dim = x.shape
    g = np.ones_like(x) if z is None else silu(z)
    g_rel = np.zeros_like(x) if z is None else silu_rel(z) + U
    v = x if norm_first else x * g
    v_rel = np.zeros_like(x) if norm_first else g_rel
    part = v.reshape(rows, groups, -1)
    m = part.shape[2]
    ms = (part ** 2).mean(-1, keepdims=True) + eps
    # Each lane adds at most ceil(m / 64) squares, then a tree of ten levels
    # joins them; the root halves the relative error, and root, reciprocal and
    # product add five roundings.
    r_rel = 0.5 * (2.0 * v_rel.max(initial=0.0) + ((m + 63) // 64 + 14) * U) + 5 * U
    out = (part / np.sqrt(ms)).reshape(rows, dim) * (1.0 if weight is None else weight)
    if norm_first:
        out = out * g
    err = np.abs(out) * (g_rel + r_rel + 4 * U)
    return out, rounded(out, err, dtype)


def verify(p, tok, u, q=None, lens=None):
    """(n_accepted, next_token, tokens): p [b,K+1,V] fp64."""
    b, rows, V = p.shape
    K = rows - 1
    p = np.where(p > 0, p, 0.0)                        # NaN and negative values count as 0
    q = None if q is None else np.where(q > 0, q, 0.0)
    n_acc, nxt = np.zeros(b, np.int32), np.zeros(b, np.int32)
    tokens = np.full((b, rows), -1, np.int32)
    for i in range(b):
        m = K if lens is None else min(max(int(lens[i]), 0), K)
        n = 0
        while n < m:
            v = tok[i, n]
            if not 0 <= v < V or not u[i, n] * (1.0 if q is None else q[i, n, v]) < p[i, n, v]:
                break
            n += 1
        r = p[i, n].copy()
        if n < m:
            if q is not None:
                r = r - q[i, n]
            elif 0 <= tok[i, n] < V:
                r[tok[i, n]] = 0.0
        r = np.where(r > 0, r, 0.0)
        if n < m and not r.any():
            r = p[i, n]
        cdf = np.cumsum(r)
        above = np.nonzero(cdf > u[i, K] * cdf[-1])[0]
        some = np.nonzero(r)[0]
        nxt[i] = above[0] if len(above) else some[-1] if len(some) else V - 1
        n_acc[i] = n
        tokens[i, :n] = tok[i, :n]
        tokens[i, n] = nxt[i]
    return n_acc, nxt, tokens

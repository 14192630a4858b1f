"""The gated delta rule and the norms between blocks in fp64 (numpy, from their
definitions), with bounds on what an fp32 evaluation with one final rounding
may differ by (U = 2^-24, see layer_refs)."""
import numpy as np

from layer_refs import HALF_STEP, U, rounded, sigmoid, silu, silu_rel


def gated_delta(q, k, v, g, beta, scale=None, l2=False, init=None, idx=None):
    """(y, final, at): q, k [b,T,G,N], v [b,T,H,P], g (or None) and beta [b,T,H]."""
    b, T, G, N = q.shape
    H, P = v.shape[2], v.shape[3]
    scale = N ** -0.5 if scale is None else scale
    if l2:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    q, k = np.repeat(q, H // G, axis=2), np.repeat(k, H // G, axis=2)
    a = np.ones((b, T, H)) if g is None else np.exp(g)
    S = np.zeros((b, H, P, N)) if init is None else init.copy()
    at = None if idx is None else S.copy()
    y = np.empty((b, T, H, P))
    for t in range(T):
        S *= a[:, t, :, None, None]
        r = v[:, t] - (S @ k[:, t, :, :, None])[..., 0]
        S += (beta[:, t, :, None] * r)[..., None] * k[:, t, :, None, :]
        y[:, t] = scale * (S @ q[:, t, :, :, None])[..., 0]
        if idx is not None:
            at[idx == t] = S[idx == t]
    return y, S, at


def delta_tolerance(N):
    """Relative bound on the fp32 states and outputs of the delta rule, in the
    2-norm over everything.  An element of the state is a decayed sum of terms
    u k; every u comes from a product over N keys' entries and at most 64
    tokens of its chunk, twice (the solution and its product), then a product
    and the decay's exponential: under N + 160 roundings, each at most U of the
    terms' size, whose sum of squares is no more than the result's times four
    (keys of norm 1, beta in [0, 1]: the update is a contraction, so errors do
    not grow from token to token)."""
    return 2.0 * (N + 160) * U


def residual_norm(x, r, w, post_norm, post_w, gate, act, layer, r_scale, b_scale, eps, dtype, stream):
    """(out, out_bound, h, h_bound): rows [rows,dim]."""
    rows, dim = x.shape
    # Roundings of a mean: each lane adds at most ceil(dim / 64) squares, then
    # a tree of ten levels joins them; root, reciprocal and product add five.
    mean_rel = 0.5 * ((dim + 63) // 64 + 14) * U + 5 * U
    n, n_rel = x, 0.0
    if post_norm:
        n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        n_rel = mean_rel
        if post_w is not None:
            n = n * post_w
            n_rel += U
    rel = np.full_like(n, n_rel)
    if gate is not None:
        f = {None: lambda v: v, "silu": silu, "sigmoid": sigmoid}[act](gate)
        rel = rel + U + (silu_rel(gate) if act else 0.0)
        n = n * f
    if layer is not None:
        n = n * layer
        rel = rel + U
    n = n * b_scale
    err = np.abs(n) * (rel + U)
    h = n
    if r is not None:
        h = r_scale * r + n
        err = err + 2 * U * (np.abs(r_scale * r) + np.abs(n))
    # h's errors move its mean square by at most 2 |h| err, averaged.
    ms = (h * h).mean(-1, keepdims=True) + eps
    ms_rel = 2 * (np.abs(h) * err).mean(-1, keepdims=True) / ms
    out = h / np.sqrt(ms) * (1.0 if w is None else w)
    factor = np.abs((1.0 if w is None else w) / np.sqrt(ms))
    out_err = factor * err + np.abs(out) * (0.5 * ms_rel + mean_rel + 3 * U)
    return out, rounded(out, out_err, dtype), h, rounded(h, err, stream)

"""Plain 64-bit implementations of pn_residual_norm and pn_logprobs with the
bounds of their fp32 arithmetic, numpy only (test helper).  Written from
include/pn.h's text."""
import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def residual_norm(h, y, post, post_gain, gate, z, scale, chan_scale, pre_gain, eps):
    """h', x in fp64 and bounds of their errors.

    h': each factor of the added term is rounded once, eight at most with the
    gate's quotient; expf is off by a step; 1 / sqrt halves the error of the
    mean, whose sum runs over 32 squares a thread, 6 steps of a wave and 16
    waves: (32 + 6 + 16) / 2 + 3.  45 U in all; the sum itself one more of h'.
    x: that error by way of the norm and of the mean (rms over rms), the
    mean's own 30 U, three roundings, and half a step of fp16."""
    h = np.asarray(h, np.float64)
    term = np.zeros_like(h)
    if y is not None:
        u = np.asarray(y, np.float64)
        if post:
            u = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
            u = u if post_gain is None else u * np.asarray(post_gain, np.float64)
        term = u * np.float64(np.float32(scale))
        if chan_scale is not None:
            term = term * np.asarray(chan_scale, np.float64)
        if gate != "none":
            z = np.asarray(z, np.float64)
            with np.errstate(over="ignore"):
                term = term * {"plain": z, "sigmoid": 1 / (1 + np.exp(-z)), "silu": z / (1 + np.exp(-z))}[gate]
    out = h + term
    dh = 45 * U * np.abs(term) + U * np.abs(out)
    mean = (out * out).mean(-1, keepdims=True)
    r = 1 / np.sqrt(mean + eps)
    g = 1.0 if pre_gain is None else np.asarray(pre_gain, np.float64)
    x = out * r * g
    lean = np.sqrt((dh * dh).mean(-1, keepdims=True)) * r
    dx = np.abs(g) * r * dh + np.abs(x) * (lean + 33 * U)
    return out, dh, x, dx + 2.0 ** -11 * (np.abs(x) + dx) + 2.0 ** -25


def clean(x):
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    return np.minimum(x, np.float64(np.finfo(np.float32).max))


def logprobs(x, scale, tokens, K):
    """ln p of tokens, entropy, top ids, their ln p, with bounds of the errors
    of ln p (without its last rounding) and of the entropy.

    exp: the difference, the constant and its product with the scale are
    rounded (3 U of the exponent), exp2 is off by 2 U, and a sum is moved to a
    larger maximum at most 20 times, 2 U each: ln S is off by (3 A + 42) U
    with A = sum p |c z|.  The entropy's sum runs over 256 entries a lane and
    the moves: 320 U of A, and the weights' own errors 3 U sum p (c z)^2."""
    x = clean(x)
    s = np.float64(np.float32(scale))
    n, V = x.shape
    top = x.max(-1, keepdims=True)
    some = top > -np.inf
    z = np.where(some, (x - np.where(some, top, 0)) * s, -np.inf)
    w = np.exp(z)
    S = w.sum(-1, keepdims=True)
    S = np.where(some, S, 1)
    lnp = np.where(some, z - np.log(S), -np.inf)
    p = w / S
    az = np.where(w > 0, -z, 0.0)
    A, B = (p * az).sum(-1), (p * az * az).sum(-1)
    H = np.where(some[:, 0], np.log(S)[:, 0] + A, 0.0)
    d_lnp = (3 * A + 42) * U
    d_H = d_lnp + (320 * A + 3 * B) * U + U * H
    tokens = np.asarray(tokens, np.int64)
    ok = (tokens >= 0) & (tokens < V)
    given = np.where(ok, np.take_along_axis(lnp, np.where(ok, tokens, 0), 1), -np.inf)
    ids = np.full((n, K), -1, np.int64)
    best = np.full((n, K), -np.inf)
    if K:
        order = np.argsort(-x, axis=-1, kind="stable")[:, :K]
        m = order.shape[1]
        live = np.take_along_axis(x, order, 1) > -np.inf
        ids[:, :m] = np.where(live, order, -1)
        best[:, :m] = np.where(live, np.take_along_axis(lnp, order, 1), -np.inf)
    return given, H, ids, best, d_lnp, d_H

"""Plain 64-bit forms of the gated delta rule and of the query/key preparation, on numpy
arrays, token by token from the definitions in include/hyb.h. Shares no code with the library.

Tolerances of the checks built on them (derived, not tuned). u = 2^-24 is fp32's rounding.
  * A state after T tokens: each token rounds every element a few times (decay, product, sum) and
    takes its correction from a sum of D products, a relative error of about sqrt(D) u / 2 of that
    correction's norm. Keys of unit length and beta <= 1 make the update a contraction, so errors of
    earlier tokens do not grow and independent ones add in squares: 2-norm of the error <=
    u sqrt(T) (4 + sqrt(D)) times the largest norm that the state had on its way.
  * An output element: |q| times the error of its state column (4 x the above, for a column's
    share may exceed the mean) times scale, plus half a step of the output's type (2^-8 relative
    for bf16). The tensor-core kernel also multiplies two-term splits of 16-bit numbers (relative
    error 2^-16 each; S, P and the corrections: at most 2^-14 together) for its outputs only.
"""
import math

import numpy as np

U = 2.0 ** -24


def bf16(x):
    """Round to nearest even, kept as float64."""
    x = np.asarray(x, np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def unit(x, eps):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps) if eps > 0 else x


def delta_rule(q, k, v, g, beta, S, scale, eps):
    """One chain of tokens of one request: q, k [T][Hk][D], v [T][Hv][D], g, beta [T][Hv],
    S [Hv][D][D]. Returns outputs, the last state, and per (token, head) the largest column
    norm of the states so far (what an error in the state is measured against)."""
    T, Hv, D = v.shape
    rep = Hv // q.shape[1]
    S = S.astype(np.float64).copy()
    out, mag = np.zeros((T, Hv, D)), np.zeros((T, Hv))
    most = np.sqrt((S * S).sum(1)).max(-1)
    norm = np.sqrt((S * S).sum((1, 2)))
    for t in range(T):
        kt = np.repeat(unit(k[t], eps), rep, axis=0)
        qt = np.repeat(unit(q[t], eps), rep, axis=0)
        S = np.exp(g[t])[:, None, None] * S
        miss = v[t] - np.einsum("hij,hi->hj", S, kt)
        S = S + kt[:, :, None] * (beta[t][:, None] * miss)[:, None, :]
        out[t] = scale * np.einsum("hij,hi->hj", S, qt)
        most = np.maximum(most, np.sqrt((S * S).sum(1)).max(-1))
        norm = np.maximum(norm, np.sqrt((S * S).sum((1, 2))))
        mag[t] = most * np.sqrt((qt * qt).sum(-1)) * abs(scale)
    return out, S, mag, norm


def state_rel(T, D):
    return U * math.sqrt(max(T, 1)) * (4 + math.sqrt(D))


def check_state(got, ref, norm, T, what):
    """got, ref [Hv][D][D]; norm [Hv]: the largest norm the state had."""
    err = np.sqrt(((got.astype(np.float64) - ref) ** 2).sum((1, 2)))
    lim = state_rel(T, ref.shape[-1]) * norm + 1e-30
    assert np.isfinite(got).all(), what
    assert (err <= lim).all(), f"{what}: error {err.max():.3e}, allowed {lim[np.argmax(err - lim)]:.3e}"


def check_out(got, ref, mag, half_step, T, what, split=False):
    """got, ref [T][Hv][D]; mag [T][Hv]; half_step of the output's type, relative."""
    assert np.isfinite(got).all(), what
    rel = 4 * state_rel(T, ref.shape[-1]) + (2.0 ** -14 if split else 0.0)
    lim = half_step * np.abs(ref) * (1 + 2 ** -8) + (rel * mag)[..., None] + 1e-30
    err = np.abs(got - ref)
    at = np.unravel_index(np.argmax(err - lim), err.shape)
    assert (err <= lim).all(), f"{what}: {err[at]:.3e} > {lim[at]:.3e} at {at}, ref {ref[at]:.3e}"


def norm_rope(x, w, w_off, eps, pos, inv_freq, m, rot, interleaved):
    """x [T][H][D] -> normed (w is not None) and rotated rows, float64."""
    x = x.astype(np.float64)
    y = x if w is None else (w.astype(np.float64) + w_off) * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = y.copy()
    if rot == 0:
        return y
    ang = pos.astype(np.float64)[:, None] * inv_freq.astype(np.float64)[None, :]
    c, s = (m * np.cos(ang))[:, None, :], (m * np.sin(ang))[:, None, :]
    if interleaved:
        a, b = y[..., 0:rot:2].copy(), y[..., 1:rot:2].copy()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :rot // 2].copy(), y[..., rot // 2:rot].copy()
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def rope_limit(x, ref, w, w_off, eps, m, rot, interleaved, half_step):
    """Allowed error of a prepared row: half a step of the type, and fp32's: the norm and weight
    take about six roundings, cos and sin are off by 2^-22 (angle and function), the turn rounds
    twice: 2^-20 of the pair's length in all."""
    x = x.astype(np.float64)
    y = x if w is None else (w.astype(np.float64) + w_off) * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    size = np.abs(y).copy()
    if rot:
        if interleaved:
            r = np.hypot(y[..., 0:rot:2], y[..., 1:rot:2])
            size[..., 0:rot:2] = size[..., 1:rot:2] = abs(m) * r
        else:
            r = np.hypot(y[..., :rot // 2], y[..., rot // 2:rot])
            size[..., :rot // 2] = size[..., rot // 2:rot] = abs(m) * r
    return half_step * np.abs(ref) * (1 + 2 ** -8) + 2.0 ** -20 * size + 1e-30

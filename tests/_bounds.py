"""Error bounds of attention outputs, derived from the arithmetic, element by element.

u is half a step of the type's rounding (bf16 2^-8, fp32 2^-24), e = 2^-24.

Weights. A score is a product of d terms summed in fp32 (any order, a factor 2 for
accumulators that truncate) and scaled: it is off by ds <= 2 (d + 2) e sum_c |q_c k_c| / sqrt(d).
A frozen logit (a + r) log2(e) is off by ds <= 4 e (|a| + |r|). The subtraction of the maximum adds
2 e |logit|, and exp (or 2^x) a relative 4 e. With s the largest of these over the row's keys,
every weight before normalisation is off by a relative w = 2 s + 8 e, and a sum of n of them
by n e more. In bf16 the weights that enter the product with V are rounded once more: u.

    o:    |do| <= (2 w + 2 n e) A + u A [bf16] + u |o|,        A = sum_j W_ij |v_j|
    lse:  |dl| <= s + 2 w + 2 n e + 8 e (|lse| + 1)

Backward (P = W from lse; dS = P (dP - D)): with x = w + n e + (u in bf16) the relative error
of a weight, and D from the stored (rounded) o,
    |d dS_ij| <= x |dS_ij| + u |dS_ij| + W_ij E_i,
    E_i = sum_c |do_c| (err(o)_ic + (d + 2) e |o_ic|) + 2 (d + 2) e max_j sum_c |do_c v_jc|
and a gradient is a sum of n terms, each with those errors, rounded once (u).
"""
import numpy as np

E = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def logit_error(q, k, a, r, i, frozen):
    """s of the module's text for the rows of one head."""
    if len(i) == 0 or k.shape[0] == 0:
        return 0.0
    d = k.shape[1]
    if frozen:
        top = int(max(i.max(), 0)) + 1
        big = np.abs(a[:k.shape[0]]).max() + np.abs(r[:top]).max()
        return 4 * E * big + 2 * E * big
    mags = np.abs(q) @ np.abs(k).T / np.sqrt(d)
    return (2 * (d + 2) * E + 2 * E) * mags.max()


def fwd(dtype, W, v, o, lse, s):
    """Bounds of o [n, d] and lse [n] of one head with weights W [n, m]."""
    n, w = W.shape[1], 2 * s + 8 * E
    A = W @ np.abs(v)
    o_tol = (2 * w + 2 * n * E) * A + HALF[dtype] * np.abs(o)
    if dtype == "bf16":
        o_tol += HALF["bf16"] * (1 + 2.0 ** -7) * A
    lse_tol = s + 2 * w + 2 * n * E + 8 * E * (np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 1)
    return o_tol + 1e-30, lse_tol


def bwd(dtype, W, q, k, v, do, o, o_tol, s):
    """Bounds (dq [n, d], dk [m, d], dv [m, d]) of one head's share."""
    n, d = W.shape[1], k.shape[1]
    u = HALF[dtype]
    x = 2 * s + 8 * E + 2 * n * E + (u if dtype == "bf16" else 0.0)
    dW = do @ v.T
    dS = np.abs(W * (dW - (W * dW).sum(axis=1, keepdims=True)))
    mags = np.abs(do) @ np.abs(v).T
    Ei = (np.abs(do) * (o_tol + (d + 2) * E * np.abs(o))).sum(axis=1) + 2 * (d + 2) * E * mags.max(axis=1)
    dS_err = (x + u + n * E) * dS + (1 + x) * W * Ei[:, None] + 2 * n * E * dS
    scale = 1 / np.sqrt(d)
    return scale * (dS_err @ np.abs(k)), scale * (dS_err.T @ np.abs(q)), (x + 2 * n * E) * (W.T @ np.abs(do))

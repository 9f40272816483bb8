"""Inputs, references and tolerances of the GPU tests of the operators over rows of logits.

Tolerances count roundings in u = 2^-24, for z = scale * x and a reference r at most 8 / log2 e
below the row's largest z (so |z_j - r| <= d_j + 6 with d_j = max z - z_j):

* a weight 2^((x - r) c): the difference, the constant c and the product err by u each of the
  exponent, 3 u ln 2 (d_j + 6) log2 e of the weight; the approximate exponent adds 4 u;
* a row's sum: the weights' errors averaged, 3 u A + 18 u + 4 u with A = sum q d, and the
  additions: a chain of at most V / 256 of them in a thread (blocks of at least 128 threads, two
  sums a thread) and 12 joins of up to 6 u each;
* log of the sum errs by that relative error, plus 2 u of its value and 2 u for the last steps:
      E = u (3 A + 100 + V / 256),
      logp: E + 4 u (|z_t - max z| + |logp| + 8),   lse: E + 4 u (|L| + 8)
* the entropy's second sum has terms q d with the errors above and one more rounding:
      E (2 + A) + 6 u sum q d^2
* a gradient's probability q_j, given L: one rounding of z - L and two of the product with log2 e,
  3 u |log q_j|, and 8 u; given the row's own sum: 3 u d_j + 26 u + E.  Terms add up, and the store
  rounds by half a step of its type, eps / 2 of the value.  The exponent flushes weights below
  2^-126 to 0: 2^-125 of the factor before them.
"""
import numpy as np
import torch

import oracle

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def to64(t):
    return t.detach().double().cpu().numpy()


def logits(rows, V, dtype, seed, spread=2.0, ld=None, offset=0):
    """[rows, V] CUDA logits in rows of ld elements, `offset` elements behind an aligned address."""
    g = torch.Generator().manual_seed(seed)
    ld = V if ld is None else ld
    flat = torch.randn(offset + rows * ld, generator=g) * spread
    return flat.to(TYPES[dtype]).cuda()[offset:].view(rows, ld)[:, :V]


def row_stats(x64, scale):
    """(max z, d, q, A, sum q d^2, E) of every row with a distribution; zeros where there is none."""
    z = scale * x64
    m = z.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        d = m - z
        q = np.exp(-d)
        q = q / q.sum(axis=1, keepdims=True)
        qd = np.where(q > 0, q * d, 0.0)
        A = qd.sum(axis=1)
        B = np.where(q > 0, qd * d, 0.0).sum(axis=1)
    E = U * (3 * A + 100 + x64.shape[1] / 256)
    return m[:, 0], d, q, A, B, E


def close(name, got, want, tol):
    """Equal where `want` is not finite, within `tol` elsewhere."""
    got, want, tol = np.broadcast_arrays(np.asarray(got, dtype=np.float64), want, tol)
    fin = np.isfinite(want)
    np.testing.assert_array_equal(got[~fin], want[~fin], err_msg=name)
    err = np.abs(np.where(fin, got, 0) - np.where(fin, want, 0))
    bad = fin & ~(err <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err, 0)), err.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} out of tolerance; worst at {i}: got "
                             f"{got[i]!r}, want {want[i]!r}, tolerance {tol[i]!r}")


def f32(v):
    """A factor as the library takes it: rounded to fp32."""
    return float(np.float32(v))


def check_logprobs(out, x64, tokens, scale, top):
    """A logprobs call's six results against the oracle."""
    scale = f32(scale)
    logp, entropy, lse, ranks, top_ids, top_logp = out
    ref = oracle.logprobs(x64, None if tokens is None else tokens.cpu().numpy(), scale, top)
    m, d, q, A, B, E = row_stats(x64, scale)
    with np.errstate(all="ignore"):
        close("lse", to64(lse), ref["lse"], E + 4 * U * (np.abs(ref["lse"]) + 8))
        if entropy is not None:
            close("entropy", to64(entropy), ref["entropy"], E * (2 + A) + 6 * U * B)
        if tokens is not None:
            t = ref["logp"]
            # z_t - max z is within log V + |logp| of 0
            size = 2 * np.abs(t) + np.log(x64.shape[1]) + 8
            close("logp", to64(logp), t, E + 4 * U * size)
        if ranks is not None:
            np.testing.assert_array_equal(ranks.cpu().numpy(), ref["ranks"])
        if top:
            np.testing.assert_array_equal(top_ids.cpu().numpy(), ref["top_ids"])
            size = 2 * np.abs(ref["top_logp"]) + np.log(x64.shape[1]) + 8
            close("top_logp", to64(top_logp), ref["top_logp"], E[:, None] + 4 * U * size)
    return ref


def tol_bwd(x64, tokens, lse, entropy, dlogp, dent, scale, want, dtype):
    with np.errstate(all="ignore"):
        logq = np.abs(scale * x64 - lse[:, None])
        q = np.exp(scale * x64 - lse[:, None])
        eq = np.where(q > 0, q * U * (3 * logq + 8), 0.0) + 2.0 ** -125
        err = np.zeros_like(x64)
        if dlogp is not None:
            hit = np.zeros_like(x64)
            ok = (tokens >= 0) & (tokens < x64.shape[1])
            hit[np.nonzero(ok)[0], tokens[ok]] = 1
            err += np.abs(dlogp)[:, None] * (eq + 4 * U * (q + hit))
        if dent is not None:
            size = np.where(q > 0, logq, 0.0) + np.abs(entropy)[:, None]
            err += np.abs(dent)[:, None] * (eq * size + q * 4 * U * size)
        err *= scale
    return err + HALF[dtype] * (np.abs(want) + err) + 2.0 ** -133


def tol_distill(x64, ids, teacher, w, scale, dloss, ref, dtype):
    """(of the losses, of the gradients)"""
    rows, V = x64.shape
    m, d, q, A, B, E = row_stats(x64, scale)
    tl, tg = np.zeros(rows), np.zeros((rows, V))
    for r in range(rows):
        kept = (ids[r] >= 0) & (ids[r] < V)
        if w[r] == 0 or not (kept & (teacher[r] != -np.inf)).any():
            continue  # nothing to learn from: 0 exactly
        with np.errstate(all="ignore"):
            u = np.where(kept, scale * teacher[r], -np.inf)
            dk = u.max() - u
            p = np.exp(-dk)
            p /= p.sum()
            Ap = np.where(p > 0, p * dk, 0).sum()
            ep = np.where(p > 0, p * U * (3 * dk + 3 * Ap + 40 + len(p) / 2), 0.0)
            dx = np.where(kept & (p > 0), np.abs(m[r] - scale * x64[r, np.clip(ids[r], 0, V - 1)]) + 6, 0.0)
            size = np.where(p > 0, dk, 0.0) + dx
            # each p_k's error meets its term; the product, the sum over up to 256 entries in a
            # tree, log P and log Z
            tl[r] = abs(w[r]) * ((ep * size).sum() + (p * size).sum() * 16 * U + E[r] + U * (3 * Ap + 60)
                                 + 4 * U * (np.log(V) + 8))
            c = abs(dloss * w[r] * scale)
            g = np.where(q[r] > 0, q[r] * (U * (3 * d[r] + 32) + E[r]), 0.0) + 2.0 ** -125
            for k in np.nonzero(kept)[0]:
                g[ids[r, k]] += ep[k] + 4 * U * p[k]
            tg[r] = c * g
    tg = tg + HALF[dtype] * (np.abs(ref["dx"]) + tg) + 2.0 ** -133
    return tl, tg

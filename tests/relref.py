"""References in 64 bits and tolerances of the tests of the softmax with a relative position bias and of
the 8-bit checkpoints.

Tolerances count roundings in u = 2^-24 (HALF of a step of the stored type comes on top):

* a score z = scale x + b (one fma) + mask errs by 2 u |z|, and the row's largest by as much of itself; the
  weight exp2((z - m) log2 e), d = m - z: difference, constant and product, 3 u d, and the approximate
  exponent 4 u: u (2 |z| + 2 |m| + 3 d + 4), of the weight;
* the row's sum: the weights' errors averaged, and its additions: at most 32 in a lane and LOOP of them for
  rows in tiles (Lk / 512), 5 in a warp, 16 warps with a factor of 8 u: 192 u + Lk / 512 u in all, which the
  reciprocal, the product and the factor of the row's own warp (8 u) are in;
* sum dy y: the same chain, ADDS = 64 + Lk / 512 of them, of |dy y|; dS = y (dy - s): y times that error, and 3 u
  of itself and of y |dy| (y |s|);
* the table's gradient: the terms' errors, and a chain of additions: an entry of a window meets each of
  a block's rows once, a lane of a far end its pairs of each row, at most 4 ceil(Lk / 256) of a row; 64 joins.
* weights below 2^-126 of the largest are flushed to 0.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def edges_of(buckets, span, both):
    """Each distance's bucket compared as whole numbers, and where it changes."""
    side = buckets // 2 if both else buckets
    near = side // 2
    far = side - near

    def bucket(n):
        if n < near:
            return n
        k = 0
        while k < far - 1 and n ** far * near ** (k + 1) >= span ** (k + 1) * near ** far:
            k += 1
        return near + k
    of = [bucket(n) for n in range(span + 1)]
    return [next(n for n, b in enumerate(of) if b >= k) for k in range(1, side)]


def buckets_of(d, edges, both):
    n = np.abs(d) if both else np.maximum(-d, 0)
    b = np.searchsorted(np.asarray(edges, dtype=np.int64), n, side="right")
    return b + (d > 0) * (len(edges) + 1) if both else b


def taking_part(B, Lq, Lk, causal, lens, q_pos):
    """([B, Lq, Lk] distances key - query, whether the key takes part)."""
    at = np.arange(Lq)[None, :, None] + (0 if q_pos is None else np.asarray(q_pos, dtype=np.int64)[:, None, None])
    d = np.broadcast_to(np.arange(Lk)[None, None, :] - at, (B, Lq, Lk))
    ok = np.ones((B, Lq, Lk), dtype=bool)
    if causal:
        ok &= d <= 0
    if lens is not None:
        ok &= np.arange(Lk)[None, None, :] < np.asarray(lens)[:, None, None]
    return d, ok


def fwd(x, table, edges, both, scale=1.0, causal=False, lens=None, q_pos=None, mask=None):
    """(y, tolerance before the store's rounding, buckets [B, Lq, Lk], kept [B, H, Lq, Lk]) of float64 arrays."""
    B, H, Lq, Lk = x.shape
    d, ok = taking_part(B, Lq, Lk, causal, lens, q_pos)
    bk = buckets_of(d, edges, both)
    z = scale * x + np.moveaxis(table[bk], 3, 1)
    kept = np.broadcast_to(ok[:, None], z.shape)
    if mask is not None:
        rows = np.arange(B * H * Lq) % mask.shape[0]
        m = mask[rows].reshape(B, H, Lq, Lk)
        kept = kept & (m != -np.inf)
        z = z + np.where(m == -np.inf, 0, m)
    z = np.where(kept, z, -np.inf)
    with np.errstate(all="ignore"):
        top = z.max(axis=3, keepdims=True)
        top = np.where(top == -np.inf, 0, top)
        e = np.exp(z - top)
        total = e.sum(axis=3, keepdims=True)
        y = np.where(kept, e / np.where(total == 0, 1, total), 0)
        far = np.where(y > 0, top - z, 0)
        rel = U * (2 * np.where(y > 0, np.abs(z), 0) + 2 * np.abs(top) + 3 * far + 4)
        tol = y * (rel + (y * rel).sum(axis=3, keepdims=True) + U * (192 + Lk / 512)) + np.where(kept, 2.0 ** -125, 0)
    return y, tol, bk, kept


def bwd(dy, y, bk, kept, buckets, scale=1.0):
    """(dx, its tolerance before the store, dtable, its tolerance before the store)."""
    B, H, Lq, Lk = dy.shape
    dy = np.where(kept & (y != 0), dy, 0)
    y = np.where(kept, y, 0)
    s = (dy * y).sum(axis=3, keepdims=True)
    es = U * (64 + Lk / 512) * (np.abs(dy * y)).sum(axis=3, keepdims=True)
    ds = y * (dy - s)
    eds = np.abs(y) * (es + 3 * U * (np.abs(dy) + np.abs(s)))
    chain = min(Lq, 128) * 4 * -(-Lk // 256) + 64
    table, tt = np.zeros((buckets, H)), np.zeros((buckets, H))
    at = np.broadcast_to(bk[:, None], ds.shape)
    for h in range(H):
        table[:, h] = np.bincount(at[:, h].ravel(), ds[:, h].ravel(), minlength=buckets)
        tt[:, h] = np.bincount(at[:, h].ravel(), (eds + chain * U * np.abs(ds))[:, h].ravel(), minlength=buckets)
    return scale * ds, abs(scale) * (eds + 2 * U * np.abs(ds)) + 2.0 ** -140, table, tt + 2.0 ** -140


def stored(tol, want, dtype):
    """The tolerance of a value stored in a type."""
    return tol + HALF[dtype] * (np.abs(want) + tol) + 2.0 ** -134


def quantise(x):
    """(q, k, values) of x [rows, cols] in 64 bits, by the definition."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    v = np.zeros((rows, blocks * 32))
    v[:, :cols] = x
    v = v.reshape(rows, blocks, 32)
    amax = np.abs(v).max(axis=2)
    k = np.full((rows, blocks), 255)
    fin = np.isfinite(amax)
    step = np.full((rows, blocks), np.nan)
    e = np.full(amax.shape, -126)
    while True:  # the least step for which the largest rounds to at most 127
        with np.errstate(all="ignore"):
            more = fin & (np.rint(amax / 2.0 ** e) > 127) & (e < 121)
        if not more.any():
            break
        e[more] += 1
    k[fin] = e[fin] + 127
    step[fin] = 2.0 ** e[fin]
    with np.errstate(all="ignore"):
        q = np.where(fin[:, :, None], np.clip(np.rint(v / step[:, :, None]), -127, 127), 0)
        values = q * step[:, :, None]
    return (q.reshape(rows, -1).astype(np.int8), k.astype(np.uint8), values.reshape(rows, -1)[:, :cols])


def norm_bwd(dy, x, gamma, mean, rstd):
    """[(value, tolerance before the store)] of dx, dgamma and, with a mean, dbeta."""
    rows, cols = dy.shape
    xhat = (x - (0 if mean is None else mean[:, None])) * rstd[:, None]
    g = dy * gamma
    n = 48 + 16  # additions of a row's sum: 32 in a lane, 5 in a warp, 16 warps; the terms' own
    a, b = g.sum(axis=1, keepdims=True), (g * xhat).sum(axis=1, keepdims=True)
    ea, eb = n * U * np.abs(g).sum(axis=1, keepdims=True), n * U * np.abs(g * xhat).sum(axis=1, keepdims=True)
    if mean is None:
        a, ea = 0 * a, 0 * ea
    r = rstd[:, None]
    dx = r * (g - (a + xhat * b) / cols)
    tol = r * (4 * U * np.abs(g) + (ea + np.abs(xhat) * eb) / cols + 6 * U * (np.abs(a) + np.abs(xhat * b)) / cols)
    chain = (rows / 152 + 24) * U  # rows of a team, the teams of a block, the joins
    out = [(dx, tol + 2 * U * np.abs(dx)), ((dy * xhat).sum(axis=0), (chain + 4 * U) * np.abs(dy * xhat).sum(axis=0))]
    if mean is not None:
        out.append((dy.sum(axis=0), chain * np.abs(dy).sum(axis=0)))
    return out


def close(name, got, want, tol):
    got = np.asarray(got, dtype=np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=name)
    with np.errstate(all="ignore"):
        bad = ~((np.abs(got - want) <= tol) | (got == want) | np.isnan(want))
    if bad.any():
        i = np.unravel_index(np.argmax(bad), bad.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} out of tolerance; first at {i}: got {got[i]!r}, want "
                             f"{np.broadcast_to(want, got.shape)[i]!r}, tolerance {np.broadcast_to(tol, got.shape)[i]!r}")


def exact_scores_tol(y, z, Lk):
    """fwd's tolerance before the store where the scores z are exact in fp32 (-inf: no key), whatever their magnitude.

    A weight's exponent is z log2 e less the product m log2 e of its warp's largest, as rounded: a rounding of at most
    1.45 (m - z) + 1 (half a step of a product below 2^25); the factor between two warps, exp2((m - top) log2 e), has two,
    of 1.45 (top - m) each: together u (2 (top - z) + 0.7) of the weight; log2 e itself is off by 0.23 u: as much of
    (top - z) again; the approximate exponent 4 u.  From 2^24 on the largest is subtracted first: two roundings of
    the differences, 2 u (top - z).  The sum's chain as in fwd, the factors of a warp (two exponents, three products) in it."""
    with np.errstate(all="ignore"):
        top = z.max(axis=3, keepdims=True)
        far = np.where(y > 0, np.where(top == -np.inf, 0, top) - z, 0)
    rel = U * (3 * far + 7)
    return y * (rel + (y * rel).sum(axis=3, keepdims=True) + U * (192 + Lk / 512)) + np.where(z > -np.inf, 2.0 ** -125, 0)

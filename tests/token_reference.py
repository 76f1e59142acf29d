"""The operators around attention over a map's tokens in 64 bits, from their
definitions, on numpy arrays, with the error bounds that the GPU tests use
(U = 2^-24; 16-bit results are rounded once more, `map_reference.stored`)."""
import numpy as np

from map_reference import ROUND, U, act, act_error, slope_error, stored, walk

TORCH = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def rounded(a, dtype):
    """The array's values as the type holds them, in float64."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, TORCH[dtype])).double().numpy()


# ---------------------------------------------------------------- linear layer
#
# A float32 sum of n products, in any order and grouping: every term passes at most
# n + 64 roundings (the last for joins of partial sums), each off by U of what is
# summed so far, below the sum of magnitudes S: (n + 64) U S.  The tensor cores
# round fewer times (once for sixteen terms), by up to 2 U where they cut.  float32
# inputs as sums of three bfloat16 values take six passes, 6 n / 16 steps of 2 U,
# and drop less than 8 U of S.

def sum_error(n, S):
    return (n + 64) * U * S


def linear(x, w, b, kind, residual=None):
    """y and z."""
    z = x @ w.T + (0 if b is None else b)
    y = act(z, kind)[0]
    return (y if residual is None else y + residual), z


def linear_bounds(x, w, b, kind, residual, dtype):
    """Bounds of y and pre."""
    y, z = linear(x, w, b, kind, residual)
    S = np.abs(x) @ np.abs(w).T
    ez = sum_error(x.shape[-1], S) + U * (np.abs(z) + (0 if b is None else np.abs(b)))
    ey = act_error(z, ez, kind) + (0 if residual is None else 2 * U * (np.abs(y) + np.abs(residual)))
    return stored(y, ey, dtype), stored(z, ez, dtype)


def linear_grad(dy, x, w, pre, kind):
    """dx, dweight, dbias, dz."""
    dz = dy if kind == "none" else dy * act(pre, kind)[1]
    K, C = w.shape
    flat = dz.reshape(-1, K)
    return dz @ w, flat.T @ x.reshape(-1, C), flat.sum(0), dz


def linear_grad_bounds(dy, x, w, pre, kind, dtype, wdtype):
    dx, dw, db, dz = linear_grad(dy, x, w, pre, kind)
    K, C = w.shape
    u, tiny = ROUND[dtype]
    e = 0 * dz if kind == "none" else np.abs(dy) * slope_error(pre, 0, kind) + U * np.abs(dz)
    # dz enters the products as a value of its type
    er = e if dtype == "f32" or kind == "none" else (1 + u) * e + u * np.abs(dz) + tiny
    P = dz.size // K
    f, fe, fr, xa = (v.reshape(-1, v.shape[-1]) for v in (np.abs(dz), e, er, np.abs(x)))
    edx = er @ np.abs(w) + sum_error(K, (np.abs(dz) + er) @ np.abs(w))
    edw = fr.T @ xa + sum_error(P, (f + fr).T @ xa)
    edb = fe.sum(0) + sum_error(min(P, 4096), f.sum(0))
    return stored(dx, edx, dtype), stored(dw, edw, wdtype), edb + U * np.abs(db)


# ------------------------------------------------- norm of queries and keys, turned

def angles(N, H, W, D, positions, base, row_pairs, col_pairs, scale):
    """(N, H, W, 1, D / 2)."""
    if positions is None:
        y, x = np.meshgrid(np.arange(H), np.arange(W), indexing="ij")
        positions = np.broadcast_to(np.stack([y, x], -1), (N, H, W, 2))
    p = positions.astype(np.longdouble)
    a = np.zeros((N, H, W, 1, D // 2), np.longdouble)
    for j in range(row_pairs):
        a[..., 0, j] = p[..., 0] * np.longdouble(scale * base ** (-j / row_pairs))
    for j in range(col_pairs):
        a[..., 0, row_pairs + j] = p[..., 1] * np.longdouble(scale * base ** (-j / col_pairs))
    return a


def step_in_turns(base, scale, j, pairs):
    """scale base^(-j / pairs) / (2 pi) as a fraction, from a hundred digits."""
    from decimal import Context, Decimal
    from fractions import Fraction
    c = Context(prec=100)
    # pi by Machin's formula
    def arc(n):
        t, s, k = Fraction(1, n), Fraction(0), 0
        while t.denominator < 10 ** 110 * max(1, t.numerator):
            s += t / (2 * k + 1) * (-1) ** k
            t /= n * n
            k += 1
        return s
    pi = 4 * (4 * arc(5) - arc(239))
    y = c.exp(c.multiply(c.ln(Decimal(base)), c.divide(Decimal(-j), Decimal(pairs))))
    return Fraction(scale) * Fraction(y) / (2 * pi)


def exact_angles(N, H, W, D, positions, base, row_pairs, col_pairs, scale):
    """`angles` for positions of any size, reduced to within half a turn before they are rounded."""
    from fractions import Fraction
    steps = [step_in_turns(base, scale, j, row_pairs) for j in range(row_pairs)]
    steps += [step_in_turns(base, scale, j, col_pairs) for j in range(col_pairs)]
    a = np.zeros((N, H, W, 1, D // 2), np.longdouble)
    for at in np.ndindex(N, H, W):
        for j, step in enumerate(steps):
            t = int(positions[at][0 if j < row_pairs else 1]) * step
            t -= round(t)
            a[at][0, j] = 2 * np.longdouble(np.pi) * np.longdouble(float(t))
    return a


def _split(v, inter):
    return (v[..., 0::2], v[..., 1::2]) if inter else (v[..., :v.shape[-1] // 2], v[..., v.shape[-1] // 2:])


def _join(a, b, inter):
    out = np.empty((*a.shape[:-1], 2 * a.shape[-1]))
    if inter:
        out[..., 0::2], out[..., 1::2] = a, b
    else:
        out[..., :a.shape[-1]], out[..., a.shape[-1]:] = a, b
    return out


def turn(v, t, inter):
    a, b = _split(v, inter)
    c, s = np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)
    return _join(a * c - b * s, a * s + b * c, inter)


def pair_sum(v, inter):
    """|a| + |b| of each pair, at both."""
    a, b = _split(np.abs(v), inter)
    return _join(a + b, a + b, inter)


def gammas(gq, gk, q, k, D):
    return np.concatenate([np.broadcast_to(g, (n, D)) for g, n in ((gq, q), (gk, k))])


def qk_norm(x, q, k, D, gq, gk, t, inter, eps):
    """(N, H, W, (q + k) D) and the bound's error before rounding."""
    v = x[..., :(q + k) * D].reshape(*x.shape[:3], q + k, D)
    r = 1 / np.sqrt((v * v).sum(-1, keepdims=True) / D + eps)
    u = v * r * gammas(gq, gk, q, k, D)
    y = turn(u, t, inter)
    # r: a sum of D squares, each term through at most D / 2 + 8 roundings of positive sums, halved by the root, and
    # the root's 2 units; the products 3; cosine and sine 6 units (angle and function), the turn 2
    err = ((D / 4 + 8) + 3 + 6 + 2) * U * pair_sum(u, inter)
    shape = (*x.shape[:3], (q + k) * D)
    return y.reshape(shape), err.reshape(shape)


def qk_norm_grad(dy, x, q, k, D, gq, gk, t, inter, eps):
    """dx of the heads, dgamma_q, dgamma_k, and their errors before rounding."""
    shape = (*x.shape[:3], q + k, D)
    v, d = (a[..., :(q + k) * D].reshape(shape) for a in (x, dy))
    g = gammas(gq, gk, q, k, D)
    r = 1 / np.sqrt((v * v).sum(-1, keepdims=True) / D + eps)
    h = v * r
    du = turn(d, -t, inter)
    w = g * du
    m = (w * v).sum(-1, keepdims=True) / D
    dx = r * w - v * r ** 3 * m
    edu = 8 * U * pair_sum(d, inter)
    ew = np.abs(g) * edu + U * np.abs(w)
    er = (D / 4 + 8) * U                       # relative
    em = (ew * np.abs(v)).sum(-1, keepdims=True) / D + (D / 2 + 10) * U * (np.abs(w * v)).sum(-1, keepdims=True) / D
    edx = r * ew + np.abs(r * w) * (er + 3 * U) + np.abs(v) * r ** 3 * em + np.abs(v * r ** 3 * m) * (3 * er + 6 * U)
    term = np.abs(du * h)
    eterm = edu * np.abs(h) + term * (er + 3 * U)
    out, outs = [], []
    for a, b in ((0, q), (q, q + k)):
        n = max(1, x.shape[0] * x.shape[1] * x.shape[2] * (b - a))
        out.append((du * h)[..., a:b, :].sum((0, 1, 2, 3)))
        outs.append(eterm[..., a:b, :].sum((0, 1, 2, 3)) + walk(n) * U * term[..., a:b, :].sum((0, 1, 2, 3)))
    flat = (*x.shape[:3], (q + k) * D)
    return dx.reshape(flat), out[0], out[1], edx.reshape(flat), outs[0], outs[1]


# ----------------------------------------------------------- relative position bias

def buckets(queries, keys, exact, side, reach, shift=0):
    """From the definition, in whole numbers: the j-th shared bucket begins at the least d with
    d^r exact^j >= exact^r reach^j."""
    r, out = side - exact, []
    for i in range(queries + keys - 1):
        d = i - (queries - 1) - shift
        m = abs(d)
        b = m
        if m >= exact:
            j = 0
            while j + 1 <= r and m ** r * exact ** (j + 1) >= exact ** r * reach ** (j + 1):
                j += 1
            b = min(side - 1, exact + j)
        out.append(side - 1 + (b if d > 0 else -b))
    return np.array(out, np.int32)


def pair_buckets(rows, cols, query, key):
    """Row and column bucket of every query and key, (queries, keys) each."""
    (qh, qw), (kh, kw) = query, key
    r = rows[np.arange(kh)[None, :] - np.arange(qh)[:, None] + qh - 1]
    c = cols[np.arange(kw)[None, :] - np.arange(qw)[:, None] + qw - 1]
    r = np.broadcast_to(r[:, None, :, None], (qh, qw, kh, kw)).reshape(qh * qw, kh * kw)
    c = np.broadcast_to(c[None, :, None, :], (qh, qw, kh, kw)).reshape(qh * qw, kh * kw)
    return r, c


def position_bias(table, rows, cols, query, key):
    """(heads, queries, keys); 0 where a bucket lies outside the table."""
    r, c = pair_buckets(rows, cols, query, key)
    ok = (r >= 0) & (r < table.shape[0]) & (c >= 0) & (c < table.shape[1])
    return np.where(ok[..., None], table[np.where(ok, r, 0), np.where(ok, c, 0)], 0.0).transpose(2, 0, 1)


def position_bias_grad(dout, rows, cols, query, key, R, C):
    """dtable (R, C, heads), the sums of magnitudes and the number of terms of a bucket."""
    r, c = pair_buckets(rows, cols, query, key)
    ok = (r >= 0) & (r < R) & (c >= 0) & (c < C)
    idx = (r * C + c)[ok]
    heads = dout.shape[1]
    out, mag = np.zeros((R * C, heads)), np.zeros((R * C, heads))
    for a in range(heads):
        for n in range(dout.shape[0]):
            v = dout[n, a][ok]
            out[:, a] += np.bincount(idx, v, R * C)
            mag[:, a] += np.bincount(idx, np.abs(v), R * C)
    count = np.bincount(idx, minlength=R * C) * dout.shape[0]
    return out.reshape(R, C, heads), mag.reshape(R, C, heads), count.reshape(R, C)

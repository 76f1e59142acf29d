"""The feature-map operators in 64 bits, from their definitions, on numpy
arrays; and the maps that the GPU tests lay them out in.

Error bounds (`*_bound`) follow float32 arithmetic with unit roundoff
U = 2^-24 and one final rounding to the map's type.
"""
import math

import numpy as np
from scipy import special

U = 2.0 ** -24
# unit roundoff, 2^-p for p significant bits (24, 8, 11), and half the smallest subnormal of the stored types
ROUND = {"f32": (2.0 ** -24, 0.0), "bf16": (2.0 ** -8, 0.0), "f16": (2.0 ** -11, 2.0 ** -25)}


def philox(counter, key):
    """Philox4x32-10 (Salmon et al., SC'11) of one counter of four words under a key of two."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p):
    return math.floor(p * 65536 + 0.5)


def drop_factor(shape, p, seed, offset, first=0):
    """0 or 65536 / (65536 - t) for each element of a map; `first`: the map's first element's number."""
    t, total = threshold(p), int(np.prod(shape))
    if t == 0:
        return np.ones(shape)
    out = np.empty(total)
    block, words = -1, None
    for i in range(total):
        e = first + i
        if e // 8 != block:
            block = e // 8
            words = philox([block & 0xFFFFFFFF, block >> 32, offset & 0xFFFFFFFF, offset >> 32],
                           [seed & 0xFFFFFFFF, seed >> 32])
        j = e % 8
        h = words[j // 2] >> 16 if j % 2 else words[j // 2] & 0xFFFF
        out[i] = 65536 / (65536 - t) if h >= t else 0.0
    return out.reshape(shape)


def act(z, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = special.expit(z)
        return z * s, s * (1 + z * (1 - s))
    if kind == "gelu":
        s = special.ndtr(z)
        return z * s, s + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return z, np.ones_like(z)


def spread(v, C):
    """(N, G) -> (N, 1, 1, C)."""
    return np.repeat(v, C // v.shape[1], axis=1)[:, None, None, :]


def group_sum(v, G):
    N, H, W, C = v.shape
    return v.reshape(N, H * W, G, C // G).sum((1, 3))


def group_norm(x, G, gamma, beta, kind, eps, factor):
    """y, mean, rstd, z."""
    N, H, W, C = x.shape
    M = H * W * C // G
    mean = group_sum(x, G) / M
    d = x - spread(mean, C)
    rstd = 1 / np.sqrt(group_sum(d * d, G) / M + eps)
    z = d * spread(rstd, C) * gamma + beta
    a = act(z, kind)[0]
    return np.where(factor == 0, 0.0, a * factor), mean, rstd, z


def group_norm_grad(dy, x, G, gamma, beta, mean, rstd, kind, factor):
    """dx, dgamma, dbeta, and dz with xh, of given mean and rstd."""
    N, H, W, C = x.shape
    M = H * W * C // G
    xh = (x - spread(mean, C)) * spread(rstd, C)
    dz = np.where(factor == 0, 0.0, dy * factor) * act(xh * gamma + beta, kind)[1]
    t = dz * gamma
    A, B = group_sum(t, G) / M, group_sum(t * xh, G) / M
    dx = spread(rstd, C) * (t - spread(A, C) - xh * spread(B, C))
    return dx, (dz * xh).sum((0, 1, 2)), dz.sum((0, 1, 2)), dz, xh


def axis_matrix(n_in, n_out):
    """(n_out, n_in): output d samples x = (d + 1/2) n_in / n_out - 1/2, taps clamped."""
    m = np.zeros((n_out, n_in))
    for d in range(n_out):
        i, r = divmod((2 * d + 1) * n_in - n_out, 2 * n_out)
        m[d, min(max(i, 0), n_in - 1)] += 1 - r / (2 * n_out)
        m[d, min(max(i + 1, 0), n_in - 1)] += r / (2 * n_out)
    return m


def resize(src, OH, OW):
    my, mx = axis_matrix(src.shape[1], OH), axis_matrix(src.shape[2], OW)
    return np.einsum("Yy,Xx,nyxc->nYXc", my, mx, src, optimize=True)


def resize_grad(ddst, H, W):
    my, mx = axis_matrix(H, ddst.shape[1]), axis_matrix(W, ddst.shape[2])
    return np.einsum("Yy,Xx,nYXc->nyxc", my, mx, ddst, optimize=True)


# ------------------------------------------------------------------ the bounds

def stored(want, err, dtype):
    """err of the float32 value plus the rounding to the map's type."""
    u, tiny = ROUND[dtype]
    return (1 + u) * err + u * np.abs(want) + tiny


def act_error(z, ez, kind):
    """Error of a float32 activation of z, itself off by ez.  Slopes stay below
    1.13.  exp is good to 2 + 1.2 |z| units, the quotient and erf to 2, and each
    of the few products and sums rounds once: below 10 + 3 |z| half-units of |z|."""
    return 1.13 * ez + (0 if kind == "none" else 1) * U * (10 + 3 * np.abs(z)) * np.abs(z)


def slope_error(z, ez, kind):
    """The same of the derivative, whose own slope stays below 1."""
    return 1.0 * ez + (0 if kind == "none" else 1) * U * (10 + 3 * np.abs(z)) * (1 + np.abs(z))


def sum_steps(terms):
    """Roundings on a term's way through the sums of a map of so many pixels:
    a thread's own run (at most terms / 1, but kernels split a run over at
    least 2 blocks of lanes once it is longer than 1024) and the joins after."""
    return min(terms, 1024) + 64


def device_map(a, dtype, pad=0, gap=0, offset=0, fill=None):
    """An (N, H, W, C) CUDA view of the array inside a flat buffer: `pad`
    elements after each row, `gap` after each image, from element `offset`; the
    rest of the buffer holds `fill`."""
    import torch
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    N, H, W, C = a.shape
    pitch = W * C + pad
    stride = H * pitch + gap
    flat = torch.full((offset + N * stride + 64,), 0.0 if fill is None else fill, dtype=dt, device="cuda")
    view = torch.as_strided(flat, (N, H, W, C), (stride, pitch, C, 1), offset)
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dt))
    return view, flat


def host(t):
    return t.detach().double().cpu().numpy()


def outside_untouched(flat, view, fill):
    """Nothing but the view's elements differs from `fill`."""
    import torch
    left = flat.clone()
    torch.as_strided(left, view.shape, view.stride(), view.storage_offset()).fill_(fill)
    return bool((left == fill).all())


def walk(terms):
    """Error of a float32 sum in units of U times the sum of magnitudes: the
    roundings on a term's way are independent, so their sum grows as a root;
    six deviations of it."""
    return 6 * math.sqrt(sum_steps(terms)) + 4


def norm_bounds(x, G, gamma, beta, kind, eps, factor, dtype):
    """Bounds of y, mean and rstd of a map held exactly."""
    N, H, W, C = x.shape
    M = H * W * C // G
    y, mean, rstd, z = group_norm(x, G, gamma, beta, kind, eps, factor)
    em = walk(M) * U * group_sum(np.abs(x), G) / M + U * np.abs(mean)
    # the variance's own sum, and the second-order effect of the mean it is taken about
    er = rstd * ((walk(M) + 10) * U / 2 + 4 * U) + 0.5 * em * em * rstd ** 3
    g = np.abs(gamma) * spread(rstd, C)
    xh = np.abs(x - spread(mean, C))
    ez = g * (spread(em, C) + 3 * U * xh) + np.abs(gamma) * xh * spread(er, C) + 2 * U * (np.abs(z) + np.abs(beta))
    ey = act_error(z, ez, kind) * factor + 2 * U * np.abs(y)
    return stored(y, ey, dtype), em, er + U * rstd


def grad_bounds(dy, x, G, gamma, beta, mean, rstd, kind, factor, dtype):
    """Bounds of dx, dgamma and dbeta of maps and statistics held exactly."""
    N, H, W, C = x.shape
    M = H * W * C // G
    dx, dgamma, dbeta, dz, xh = group_norm_grad(dy, x, G, gamma, beta, mean, rstd, kind, factor)
    z = xh * gamma + beta
    exh = 3 * U * np.abs(xh)
    ez = np.abs(gamma) * exh + 2 * U * (np.abs(z) + np.abs(beta))
    edz = np.abs(dy * factor) * slope_error(z, ez, kind) + 3 * U * np.abs(dz)
    eb = edz.sum((0, 1, 2)) + walk(N * H * W) * U * np.abs(dz).sum((0, 1, 2)) + U * np.abs(dbeta)
    eg = ((edz * np.abs(xh) + np.abs(dz) * exh).sum((0, 1, 2)) + U * np.abs(dgamma)
          + walk(N * H * W) * U * np.abs(dz * xh).sum((0, 1, 2)))
    ag, at = np.abs(gamma) * edz, np.abs(gamma * dz)
    A, B = group_sum(gamma * dz, G) / M, group_sum(gamma * dz * xh, G) / M
    eA = group_sum(ag, G) / M + walk(M) * U * group_sum(at, G) / M
    eB = group_sum(ag * np.abs(xh) + at * 3 * U * np.abs(xh), G) / M + walk(M) * U * group_sum(at * np.abs(xh), G) / M
    A, B, eA, eB = (spread(np.abs(v), C) for v in (A, B, eA, eB))
    edx = spread(rstd, C) * (ag + eA + exh * B + np.abs(xh) * eB + 4 * U * (at + A + np.abs(xh) * B))
    return stored(dx, edx, dtype), eg, eb

"""The feature-map operators in measured form: group norm with an activation,
dropout from a counter, and the bilinear resize of maps and position tables,
each with its gradient.

Maps are channels last, (N, H, W, C).  ``run`` is one call of an operator:
in plain torch operations on 32-bit floats where ``own`` is false, through
the package's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
#: No drawn case has more map elements than this (the largest listed ones have as many).
_MOST = 134217728


# ---------------------------------------------------------------- the cases

def _norm(name, op, n, h, w, c, g, dtype, act, p):
    return {"name": name, "op": op, "n": n, "h": h, "w": w, "c": c, "groups": g, "dtype": dtype, "act": act, "p": p}


def _drop(name, n, h, w, c, dtype, p, residual):
    return {"name": name, "op": "dropout", "n": n, "h": h, "w": w, "c": c, "dtype": dtype, "p": p,
            "residual": residual}


def _map(name, op, n, h, w, oh, ow, c, dtype, table, src_dtype):
    return {"name": name, "op": op, "n": n, "h": h, "w": w, "oh": oh, "ow": ow, "c": c, "dtype": dtype,
            "table": table, "src_dtype": src_dtype}


def listed():
    return [
        # one pair of small maps through a deep stage of an encoder: the launch is what it costs
        _norm("norm_small", "norm", 2, 14, 14, 256, 32, "bf16", "silu", 0.0),
        # a training batch through a middle stage, norm -> SiLU -> dropout in one call; 10 channels a group
        _norm("norm_train", "norm", 16, 64, 64, 320, 32, "bf16", "silu", 0.1),
        # the last stage of a decoder at 512 x 512: few channels, each sample larger than any on-chip memory
        _norm("norm_large", "norm", 4, 512, 512, 128, 32, "bf16", "silu", 0.0),
        # the gradient in full precision on an odd image size
        _norm("norm_grad_ragged", "norm_grad", 3, 37, 53, 96, 8, "f32", "gelu", 0.0),
        # the gradient of a training batch's wide stage, with the dropout mask made again
        _norm("norm_grad_large", "norm_grad", 8, 128, 128, 512, 32, "bf16", "silu", 0.1),
        # one image's tokens, or the gradient of them: the launch is what it costs
        _drop("dropout_small", 1, 14, 14, 384, "f32", 0.1, False),
        # an odd batch of odd maps added to the block's input
        _drop("dropout_ragged", 7, 61, 83, 200, "f16", 0.25, True),
        # a large training batch added to the block's input
        _drop("dropout_large", 32, 64, 64, 1024, "bf16", 0.1, True),
        # a learned 24 x 24 position table brought to the grid of a batch of wide images and added to their tokens
        _map("table_add", "resize", 16, 24, 24, 37, 50, 1024, "bf16", True, "f32"),
        # the gradient of that table, summed over the batch
        _map("table_grad", "resize_grad", 16, 24, 24, 37, 50, 1024, "bf16", True, "f32"),
        # the upsampling between two stages of a decoder
        _map("upsample", "resize", 8, 128, 128, 256, 256, 256, "bf16", False, "bf16"),
        # and its gradient
        _map("upsample_grad", "resize_grad", 8, 128, 128, 256, 256, 256, "f16", False, "f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm", "norm_grad", "dropout", "resize", "resize_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    p = rng.choice([0.0, 0.0, 0.1, round(rng.uniform(0.02, 0.6), 3)])
    while True:
        n, h, w = _log(rng, 1, 32), _log(rng, 4, 512), _log(rng, 4, 512)
        if op in ("norm", "norm_grad"):
            g = rng.choice([4, 8, 16, 32, 32, 32])
            c = g * _log(rng, 2, 32)
            limit = _MOST // (4 if dtype == "f32" else 2) if op == "norm_grad" else _MOST // (2 if dtype == "f32" else 1)
            if 4096 <= n * h * w * c <= limit:
                return _norm("", op, n, h, w, c, g, dtype, rng.choice(["none", "silu", "silu", "gelu"]), p)
        elif op == "dropout":
            c = rng.choice([_log(rng, 1, 2048), 8 * _log(rng, 1, 256)])
            if 4096 <= n * h * w * c <= _MOST // (2 if dtype == "f32" else 1):
                return _drop("", n, h, w, c, dtype, max(p, 0.05), rng.random() < 0.5)
        else:
            table = rng.random() < 0.5
            if table:
                h, w = _log(rng, 4, 64), _log(rng, 4, 64)
            oh = max(1, round(h * math.exp(rng.uniform(math.log(0.4), math.log(3.0)))))
            ow = max(1, round(w * math.exp(rng.uniform(math.log(0.4), math.log(3.0)))))
            c = rng.choice([_log(rng, 1, 2048), 8 * _log(rng, 1, 256)])
            limit = _MOST // (8 if dtype == "f32" else 4)
            if max(n * oh * ow * c, n * h * w * c) <= limit and 4096 <= n * oh * ow * c:
                return _map("", op, n, h, w, oh, ow, c, dtype, table, rng.choice(["f32", dtype]) if table else dtype)


def work(case):
    es = _SIZE[case["dtype"]]
    n, h, w, c = case["n"], case["h"], case["w"], case["c"]
    e = n * h * w * c
    if case["op"] == "norm":
        return {"bytes": 2 * e * es + 8 * c + 8 * n * case["groups"], "flops": 12 * e}
    if case["op"] == "norm_grad":
        return {"bytes": 3 * e * es + 16 * c + 8 * n * case["groups"], "flops": 24 * e}
    if case["op"] == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * e * es, "flops": 2 * e}
    e, o, ss = (1 if case["table"] else n) * h * w * c, n * case["oh"] * case["ow"] * c, _SIZE[case["src_dtype"]]
    if case["op"] == "resize":
        return {"bytes": e * ss + (2 if case["table"] else 1) * o * es, "flops": (7 if case["table"] else 6) * o}
    return {"bytes": e * ss + o * es, "flops": 8 * o}


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    dt = _TYPES[case["dtype"]]
    n, h, w, c = case["n"], case["h"], case["w"], case["c"]
    st = {"case": case, "dtype": dt, "seed": (seed * 2654435761 + 12345) % (1 << 62), "offset": seed % 1009}
    if case["op"] in ("norm", "norm_grad"):
        g = case["groups"]
        # features after a convolution: every channel has a scale and an offset of its own
        x = normal(n, h, w, c)
        x *= 0.5 + torch.rand(c, device=dev, generator=gen)
        x += 0.5 * normal(c)
        st["x"] = x.to(dt)
        st["gamma"] = 1.0 + 0.2 * normal(c)
        st["beta"] = 0.2 * normal(c)
        if case["op"] == "norm":
            st["y"] = torch.empty_like(st["x"])
            st["mean"] = torch.empty((n, g), device=dev)
            st["rstd"] = torch.empty((n, g), device=dev)
        else:
            del x
            v = st["x"].float().view(n, h * w, g, c // g)
            st["mean"] = v.mean((1, 3))
            st["rstd"] = torch.rsqrt((v - st["mean"][:, None, :, None]).square().mean((1, 3)) + EPS)
            del v
            st["dy"] = normal(n, h, w, c).to(dt)
            st["dx"] = torch.empty_like(st["x"])
            st["dgamma"] = torch.empty(c, device=dev)
            st["dbeta"] = torch.empty(c, device=dev)
    elif case["op"] == "dropout":
        st["x"] = normal(n, h, w, c).to(dt)
        st["residual"] = normal(n, h, w, c).to(dt) if case["residual"] else None
        st["y"] = torch.empty_like(st["x"])
    else:
        sd, oh, ow = _TYPES[case["src_dtype"]], case["oh"], case["ow"]
        ns = 1 if case["table"] else n
        if case["op"] == "resize":
            st["src"] = normal(ns, h, w, c).to(sd)
            st["base"] = normal(n, oh, ow, c).to(dt) if case["table"] else None
            st["dst"] = torch.empty((n, oh, ow, c), dtype=dt, device=dev)
        else:
            st["ddst"] = normal(n, oh, ow, c).to(dt)
            st["dsrc"] = torch.empty((ns, h, w, c), dtype=sd, device=dev)
        # the sampling of each axis: near tap, far tap and the far tap's weight
        st["ys"], st["xs"] = _axis(h, oh, dev), _axis(w, ow, dev)
    return st


def _axis(n_in, n_out, dev):
    d = torch.arange(n_out, device=dev, dtype=torch.int64)
    num, den = (2 * d + 1) * n_in - n_out, 2 * n_out
    i = torch.div(num, den, rounding_mode="floor")
    u = ((num - i * den).double() / den).float()
    return i.clamp(0, n_in - 1), (i + 1).clamp(0, n_in - 1), u


# ----------------------------------------------------------- the plain form

def _mulhilo(a, b):
    """High and low 32 bits of the product of 32-bit values held in int64."""
    lo16, hi16 = b & 0xFFFF, b >> 16
    low = a * lo16
    mid = a * hi16 + (low >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (low & 0xFFFF)


def _keep(total, p, seed, offset, dev):
    """The kept elements of a map of `total`: Philox4x32-10 (Salmon et al.,
    "Parallel random numbers: as easy as 1, 2, 3") on the counter
    (element / 8, offset) under the key `seed`, 16 bits an element."""
    i = torch.arange((total + 7) // 8, device=dev, dtype=torch.int64)
    c0, c1 = i & 0xFFFFFFFF, i >> 32
    c2, c3 = torch.full_like(i, offset & 0xFFFFFFFF), torch.full_like(i, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack((c0, c1, c2, c3), 1)
    halves = torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:total]
    return halves >= _threshold(p)


def _threshold(p):
    return int(p * 65536 + 0.5)


def _dropped(x, p, seed, offset):
    t = _threshold(p)
    if t == 0:
        return x
    keep = _keep(x.numel(), p, seed, offset, x.device).view(x.shape)
    return torch.where(keep, x * (65536 / (65536 - t) if t < 65536 else 0.0), torch.zeros((), device=x.device))


def _phi(z):
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z * _phi(z) if act == "gelu" else z


def _act_slope(z, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return _phi(z) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    return torch.ones((), device=z.device)


def _plain_norm(st):
    c = st["case"]
    n, h, w, ch, g = c["n"], c["h"], c["w"], c["c"], c["groups"]
    v = st["x"].float().view(n, h * w, g, ch // g)
    mean = v.mean((1, 3))
    v = v - mean[:, None, :, None]
    rstd = torch.rsqrt(v.square().mean((1, 3)) + EPS)
    z = (v * rstd[:, None, :, None]).view(n, h, w, ch) * st["gamma"] + st["beta"]
    y = _dropped(_act(z, c["act"]), c["p"], st["seed"], st["offset"])
    return {"y": y.to(st["dtype"]), "mean": mean, "rstd": rstd}


def _plain_norm_grad(st):
    c = st["case"]
    n, h, w, ch, g = c["n"], c["h"], c["w"], c["c"], c["groups"]
    v = st["x"].float().view(n, h * w, g, ch // g)
    xh = ((v - st["mean"][:, None, :, None]) * st["rstd"][:, None, :, None]).view(n, h, w, ch)
    dz = _dropped(st["dy"].float(), c["p"], st["seed"], st["offset"]) * _act_slope(xh * st["gamma"] + st["beta"], c["act"])
    dbeta, dgamma = dz.sum((0, 1, 2)), (dz * xh).sum((0, 1, 2))
    t = (dz * st["gamma"]).view(v.shape)
    xh = xh.view(v.shape)
    a, b = t.mean((1, 3), keepdim=True), (t * xh).mean((1, 3), keepdim=True)
    dx = (t - a - xh * b) * st["rstd"][:, None, :, None]
    return {"dx": dx.view(n, h, w, ch).to(st["dtype"]), "dgamma": dgamma, "dbeta": dbeta}


def _plain_dropout(st):
    y = _dropped(st["x"].float(), st["case"]["p"], st["seed"], st["offset"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.to(st["dtype"])}


def _plain_resize(st):
    (y0, y1, v), (x0, x1, u) = st["ys"], st["xs"]
    s = st["src"].float()
    u, v = u[:, None], v[:, None, None]
    s = s[:, :, x0] * (1.0 - u) + s[:, :, x1] * u
    s = s[:, y0] * (1.0 - v) + s[:, y1] * v
    if st["base"] is not None:
        s = s + st["base"].float()
    return {"dst": s.to(st["dtype"])}


def _plain_resize_grad(st):
    (y0, y1, v), (x0, x1, u) = st["ys"], st["xs"]
    c = st["case"]
    d = st["ddst"].float()
    if c["table"]:
        d = d.sum(0, keepdim=True)
    u, v = u[:, None], v[:, None, None]
    rows = torch.zeros((d.shape[0], c["h"], c["ow"], c["c"]), device=d.device)
    rows.index_add_(1, y0, d * (1.0 - v))
    rows.index_add_(1, y1, d * v)
    out = torch.zeros((d.shape[0], c["h"], c["w"], c["c"]), device=d.device)
    out.index_add_(2, x0, rows * (1.0 - u))
    out.index_add_(2, x1, rows * u)
    return {"dsrc": out.to(st["dsrc"].dtype)}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dropout": _plain_dropout, "resize": _plain_resize,
          "resize_grad": _plain_resize_grad}


# ------------------------------------------------------ the framework's calls

def _own(st):
    import bilinear_image_resize_gb300 as rz
    c = st["case"]
    if c["op"] in ("norm", "norm_grad"):
        act = {"none": rz.RZ_ACT_NONE, "silu": rz.RZ_ACT_SILU, "gelu": rz.RZ_ACT_GELU}[c["act"]]
        drop = (c["p"], st["seed"], st["offset"]) if c["p"] else None
    if c["op"] == "norm":
        rz.map_group_norm(st["x"], st["y"], c["groups"], st["gamma"], st["beta"], st["mean"], st["rstd"], act=act,
                          eps=EPS, drop=drop)
        return {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    if c["op"] == "norm_grad":
        rz.map_group_norm_grad(st["dy"], st["x"], st["dx"], c["groups"], st["gamma"], st["beta"], st["mean"],
                               st["rstd"], st["dgamma"], st["dbeta"], act=act, drop=drop)
        return {"dx": st["dx"], "dgamma": st["dgamma"], "dbeta": st["dbeta"]}
    if c["op"] == "dropout":
        rz.map_dropout(st["x"], st["y"], c["p"], st["seed"], st["offset"], residual=st["residual"])
        return {"y": st["y"]}
    if c["op"] == "resize":
        rz.resize_map(st["src"], st["dst"], base=st["base"])
        return {"dst": st["dst"]}
    rz.resize_map_grad(st["ddst"], st["dsrc"])
    return {"dsrc": st["dsrc"]}


def run(st):
    return _own(st) if own else _PLAIN[st["case"]["op"]](st)


# -------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    def kept(total, p, seed, offset):
        """The kept elements again, on the host with 64-bit products, and what they are multiplied by."""
        t = int(math.floor(p * 65536 + 0.5))
        keep = np.empty((total + 7) // 8 * 8, np.bool_)
        word = np.uint64(0xFFFFFFFF)
        for at in range(0, len(keep) // 8, 1 << 20):
            i = np.arange(at, min(at + (1 << 20), len(keep) // 8), dtype=np.uint64)
            ctr = [i & word, i >> np.uint64(32), np.full_like(i, offset % 2 ** 32), np.full_like(i, offset // 2 ** 32)]
            key = [seed % 2 ** 32, seed // 2 ** 32]
            for _ in range(10):
                a, b = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
                ctr = [(b >> np.uint64(32)) ^ ctr[1] ^ np.uint64(key[0]), b & word,
                       (a >> np.uint64(32)) ^ ctr[3] ^ np.uint64(key[1]), a & word]
                key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
            bits = np.stack([v.astype("<u4") for v in ctr], 1).view("<u2")
            keep[8 * at:8 * (at + len(i))] = (bits >= t).reshape(-1)
        return keep[:total], (0.0 if t == 65536 else 65536.0 / (65536 - t))

    def weights(n_in, n_out):
        """The (n_out, n_in) matrix of one axis."""
        m = np.zeros((n_out, n_in))
        for d in range(n_out):
            i, r = divmod((2 * d + 1) * n_in - n_out, 2 * n_out)
            m[d, min(max(i, 0), n_in - 1)] += 1 - r / (2 * n_out)
            m[d, min(max(i + 1, 0), n_in - 1)] += r / (2 * n_out)
        return torch.from_numpy(m).to(dev)

    if case["op"] in ("norm", "norm_grad", "dropout"):
        elements = case["n"] * case["h"] * case["w"] * case["c"]
        if case["p"] and elements > _MOST:
            return None
    st = prepare(case, seed)
    dev, f = "cuda", torch.float64
    n, h, w, c = case["n"], case["h"], case["w"], case["c"]
    factor = None
    if case["op"] in ("norm", "norm_grad", "dropout") and case["p"]:
        keep, scale = kept(elements, case["p"], st["seed"], st["offset"])
        factor = torch.from_numpy(keep).to(dev).view(n, h, w, c).to(f).mul_(scale)
    if case["op"] == "dropout":
        y = st["x"].to(f) * factor
        return {"y": y if st["residual"] is None else y + st["residual"].to(f)}
    if case["op"] in ("norm", "norm_grad"):
        g = case["groups"]
        gamma, beta = st["gamma"].to(f), st["beta"].to(f)

        def slopes(z):
            """The activation and its derivative."""
            if case["act"] == "silu":
                s = torch.sigmoid(z)
                return z * s, s + z * s * (1 - s)
            if case["act"] == "gelu":
                s = torch.special.ndtr(z)
                return z * s, s + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
            return z, torch.ones_like(z)

        def grouped(v):
            return v.reshape(h * w, g, c // g).transpose(0, 1).reshape(g, -1)

        def back(v):
            return v.reshape(g, h * w, c // g).transpose(0, 1).reshape(h, w, c)

        outs, means, rstds, dgamma, dbeta = [], [], [], torch.zeros(c, dtype=f, device=dev), torch.zeros(c, dtype=f, device=dev)
        for k in range(n):
            x = grouped(st["x"][k].to(f))
            if case["op"] == "norm":
                var, mean = torch.var_mean(x, 1, correction=0)
                rstd = 1 / torch.sqrt(var + EPS)
                y = slopes(back((x - mean[:, None]) * rstd[:, None]) * gamma + beta)[0]
                outs.append(y if factor is None else y * factor[k])
                means.append(mean)
                rstds.append(rstd)
            else:
                rstd = st["rstd"][k].to(f)[:, None]
                xh = back((x - st["mean"][k].to(f)[:, None]) * rstd)
                dz = st["dy"][k].to(f) * slopes(xh * gamma + beta)[1]
                if factor is not None:
                    dz = dz * factor[k]
                dbeta += dz.sum((0, 1))
                dgamma += (dz * xh).sum((0, 1))
                t, xh = grouped(dz * gamma), grouped(xh)
                outs.append(back(rstd * (t - t.mean(1, True) - xh * (t * xh).mean(1, True))))
        if case["op"] == "norm":
            return {"y": torch.stack(outs), "mean": torch.stack(means), "rstd": torch.stack(rstds)}
        return {"dx": torch.stack(outs), "dgamma": dgamma, "dbeta": dbeta}
    my, mx = weights(h, case["oh"]), weights(w, case["ow"])
    if case["op"] == "resize":
        s = torch.einsum("Yy,nyxc->nYxc", my, st["src"].to(f))
        s = torch.einsum("Xx,nYxc->nYXc", mx, s)
        return {"dst": s.expand(n, -1, -1, -1) if st["base"] is None else s + st["base"].to(f)}
    d = st["ddst"].to(f)
    if case["table"]:
        d = d.sum(0, keepdim=True)
    return {"dsrc": torch.einsum("Yy,nYxc->nyxc", my, torch.einsum("Xx,nYXc->nYxc", mx, d))}

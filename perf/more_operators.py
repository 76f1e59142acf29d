"""The operators around attention over a feature map's tokens in measured form:
the linear layer with its epilogue, the norm of queries and keys with the
position rotation, and the relative position bias by buckets, each with its
gradient.

Maps are channels last, (N, H, W, C); scores are (N, heads, queries, keys).
``run`` is one call of an operator: in plain torch operations on 32-bit floats
where ``own`` is false, through the package's entry points where it is true.
"""
import math

import torch

own = False

EPS = 1e-6
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
#: No drawn case does more than the largest listed ones: products, and elements of a map or of scores.
_MOST_FLOPS = 2 * 65536 * 1024 * 4096
_MOST_MAP = 12 * 64 * 64 * 2560
_MOST_SCORES = 16 * 4096 * 4096


# ---------------------------------------------------------------- the cases

def _linear(name, op, n, h, w, c, k, dtype, act, residual=False):
    return {"name": name, "op": op, "n": n, "h": h, "w": w, "c": c, "k": k, "dtype": dtype, "act": act,
            "residual": residual}


def _qk(name, op, n, h, w, q_heads, k_heads, v_heads, d, dtype, base, row_pairs, col_pairs, interleaved, far):
    return {"name": name, "op": op, "n": n, "h": h, "w": w, "q_heads": q_heads, "k_heads": k_heads, "v_heads": v_heads,
            "d": d, "dtype": dtype, "base": base, "row_pairs": row_pairs, "col_pairs": col_pairs,
            "interleaved": interleaved, "far": far}


def _bias(name, op, n, heads, qh, qw, kh, kw, oy, ox, dtype, exact_to, side, reach, scores):
    return {"name": name, "op": op, "n": n, "heads": heads, "qh": qh, "qw": qw, "kh": kh, "kw": kw, "oy": oy, "ox": ox,
            "dtype": dtype, "exact": exact_to, "side": side, "reach": reach, "scores": scores}


def listed():
    return [
        # one token through the first product of an MLP, as it is served: the weights are all there is to read
        _linear("linear_token", "linear", 1, 1, 1, 1024, 4096, "bf16", "gelu"),
        # a projection in full precision on an odd batch, odd map and odd width, added to the block's input
        _linear("linear_ragged", "linear", 3, 37, 53, 96, 250, "f32", "silu", True),
        # the projection after attention for a batch of 24 x 24 grids, added to the block's input
        _linear("linear_block", "linear", 16, 24, 24, 1024, 1024, "f16", "none", True),
        # the first product of an MLP for a large batch of 64 x 64 grids
        _linear("linear_large", "linear", 16, 64, 64, 1024, 4096, "bf16", "gelu"),
        # the gradient of a small layer whose widths fill no tile
        _linear("linear_grad_ragged", "linear_grad", 7, 13, 17, 200, 322, "f16", "gelu"),
        # the gradient of a training batch's layer
        _linear("linear_grad", "linear_grad", 8, 64, 64, 1024, 1024, "bf16", "silu"),
        # the next token of eight long sequences with shared key heads: far positions, a launch is what it costs
        _qk("qk_token", "qk_norm", 8, 1, 1, 16, 4, 4, 128, "bf16", 500000.0, 0, 64, False, True),
        # queries and keys of a training batch's 64 x 64 grids, half of the pairs turned by row, half by column
        _qk("qk_large", "qk_norm", 12, 64, 64, 20, 20, 20, 64, "bf16", 100.0, 16, 16, False, False),
        # the gradient of queries with fewer key heads on a wide odd grid, neighbouring elements as pairs
        _qk("qk_grad", "qk_norm_grad", 16, 37, 50, 16, 4, 4, 128, "f16", 100.0, 32, 32, True, False),
        # scores of many 7 x 7 windows, padding masked: every offset has a bucket of its own
        _bias("bias_windows", "bias", 1024, 8, 7, 7, 7, 7, 0, 0, "f16", 7, 7, 8, True),
        # the bias of a 64 x 64 grid, made once for a batch's attention; far offsets share buckets
        _bias("bias_large", "bias", 1, 16, 64, 64, 64, 64, 0, 0, "bf16", 8, 16, 64, False),
        # the gradient of the table over a batch of wide odd grids
        _bias("bias_grad", "bias_grad", 4, 12, 37, 50, 37, 50, 0, 0, "bf16", 4, 12, 40, True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "qk_norm", "qk_norm_grad", "bias", "bias_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    wide = dtype == "f32"
    while True:
        n, h, w = _log(rng, 1, 32), _log(rng, 1, 128), _log(rng, 1, 128)
        if op in ("linear", "linear_grad"):
            if rng.random() < 0.25:
                h = w = 1
            c, k = (rng.choice([_log(rng, 1, 4096), 8 * _log(rng, 1, 512)]) for _ in range(2))
            flops, p = (4 if op == "linear_grad" else 2) * n * h * w * c * k, n * h * w
            if 4096 <= flops <= _MOST_FLOPS // (8 if wide else 1) and p * max(c, k) <= _MOST_SCORES // (2 if wide else 1):
                return _linear("", op, n, h, w, c, k, dtype, rng.choice(["none", "silu", "gelu"]),
                               op == "linear" and rng.random() < 0.5)
        elif op in ("qk_norm", "qk_norm_grad"):
            kh = _log(rng, 1, 20)
            qh, vh = kh * rng.choice([1, 1, 2, 4, 8]), rng.choice([0, kh])
            d = rng.choice([32, 64, 64, 128, 256, 2 * _log(rng, 2, 128)])
            rows = rng.choice([0, d // 4, rng.randrange(0, d // 2 + 1)])
            cols = rng.choice([d // 2 - rows, rng.randrange(0, d // 2 - rows + 1)])
            limit = _MOST_MAP // (2 if wide else 1) // (2 if op == "qk_norm_grad" else 1)
            if 1024 <= n * h * w * (qh + kh) * d <= limit:
                return _qk("", op, n, h, w, qh, kh, vh, d, dtype, rng.choice([100.0, 10000.0, 500000.0]), rows, cols,
                           rng.random() < 0.5, rng.random() < 0.5)
        else:
            n, heads = _log(rng, 1, 1024), _log(rng, 1, 32)
            kh, kw = _log(rng, 1, 64), _log(rng, 1, 64)
            kind, oy, ox = rng.random(), 0, 0
            if kind < 0.2:       # one query somewhere in the grid
                qh, qw, oy, ox = 1, 1, rng.randrange(kh), rng.randrange(kw)
            elif kind < 0.4:     # a sequence
                kh, kw = _log(rng, 1, 4096), 1
                qh, qw = kh, 1
            else:
                qh, qw = kh, kw
            exact_to = _log(rng, 1, 16)
            side = exact_to + rng.choice([0, _log(rng, 1, 16)])
            scores = op == "bias_grad" or rng.random() < 0.6
            total = (n if scores else 1) * heads * qh * qw * kh * kw
            if 4096 <= total <= _MOST_SCORES // ((2 if wide else 1) * (2 if scores else 1)):
                return _bias("", op, n if scores else 1, heads, qh, qw, kh, kw, oy, ox, dtype, exact_to, side,
                             side + _log(rng, 1, 128), scores)


def work(case):
    es = _SIZE[case["dtype"]]
    op = case["op"]
    if op in ("linear", "linear_grad"):
        p, c, k = case["n"] * case["h"] * case["w"], case["c"], case["k"]
        if op == "linear":
            return {"bytes": es * (p * c + k * c + p * k * (2 if case["residual"] else 1)) + 4 * k, "flops": 2 * p * c * k}
        return {"bytes": es * (2 * p * c + 2 * k * c + p * k * (1 if case["act"] == "none" else 2)) + 4 * k,
                "flops": 4 * p * c * k}
    if op in ("qk_norm", "qk_norm_grad"):
        p = case["n"] * case["h"] * case["w"]
        e = p * (case["q_heads"] + case["k_heads"]) * case["d"]
        at = 8 * p if case["far"] else 0
        if op == "qk_norm":
            return {"bytes": 2 * e * es + 8 * case["d"] + at, "flops": 8 * e}
        return {"bytes": 3 * e * es + 16 * case["d"] + at, "flops": 16 * e}
    s = 2 * case["side"] - 1
    e, t = case["n"] * case["heads"] * case["qh"] * case["qw"] * case["kh"] * case["kw"], 4 * s * s * case["heads"]
    return {"bytes": e * es * (2 if op == "bias" and case["scores"] else 1) + t, "flops": e}


# --------------------------------------------------------------- the inputs

def _buckets(queries, keys, offset, exact_to, side, reach):
    """The bucket of every offset of an axis, from key 0 - query `queries` - 1 to key `keys` - 1 - query 0: offsets up
    to `exact_to` have one of their own, those up to `reach` share `side` - `exact_to` in steps that grow as a power."""
    starts, r = [], side - exact_to
    for j in range(1, r):        # the least d with log(d / exact) / log(reach / exact) r >= j
        lo, hi = exact_to, reach
        while lo < hi:
            d = (lo + hi) // 2
            if d ** r * exact_to ** j >= exact_to ** r * reach ** j:
                hi = d
            else:
                lo = d + 1
        starts.append(lo)
    out = []
    for i in range(queries + keys - 1):
        d = i - (queries - 1) - offset
        b = abs(d) if abs(d) < exact_to else min(side - 1, exact_to + sum(abs(d) >= s for s in starts))
        out.append(side - 1 + (b if d >= 0 else -b))
    return out


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    op, dt = case["op"], _TYPES[case["dtype"]]
    st = {"case": case, "dtype": dt}
    if op in ("linear", "linear_grad"):
        n, h, w, c, k = case["n"], case["h"], case["w"], case["c"], case["k"]
        st["x"] = normal(n, h, w, c).to(dt)
        st["weight"] = (normal(k, c) * c ** -0.5).to(dt)
        st["bias"] = 0.2 * normal(k)
        if op == "linear":
            st["residual"] = normal(n, h, w, k).to(dt) if case["residual"] else None
            st["y"] = torch.empty((n, h, w, k), dtype=dt, device=dev)
        else:
            st["dy"] = normal(n, h, w, k).to(dt)
            # what the forward call left of the values before the activation
            st["pre"] = None if case["act"] == "none" else (st["x"].float() @ st["weight"].float().t() + st["bias"]).to(dt)
            st["dx"] = torch.empty_like(st["x"])
            st["dweight"] = torch.empty_like(st["weight"])
            st["dbias"] = torch.empty(k, device=dev)
    elif op in ("qk_norm", "qk_norm_grad"):
        n, h, w, d = case["n"], case["h"], case["w"], case["d"]
        qk = (case["q_heads"] + case["k_heads"]) * d
        # what a projection leaves: every channel has a scale of its own
        c = qk + case["v_heads"] * d
        st["x"] = (normal(n, h, w, c) * (0.5 + torch.rand(c, device=dev, generator=gen))).to(dt)
        st["gamma_q"], st["gamma_k"] = 1.0 + 0.2 * normal(d), 1.0 + 0.2 * normal(d)
        st["positions"] = (torch.randint(0, 1 << 20, (n, h, w, 2), device=dev, generator=gen, dtype=torch.int32)
                           if case["far"] else None)
        if op == "qk_norm":
            st["y"] = torch.empty((n, h, w, qk), dtype=dt, device=dev)
        else:
            st["dy"] = normal(n, h, w, qk).to(dt)
            st["dx"] = torch.zeros_like(st["x"])     # of the query, key and value channels; the last are attention's to write
            st["dgamma_q"], st["dgamma_k"] = torch.empty(d, device=dev), torch.empty(d, device=dev)
    else:
        n, heads = case["n"], case["heads"]
        lq, lk, s = case["qh"] * case["qw"], case["kh"] * case["kw"], 2 * case["side"] - 1
        rule = (case["exact"], case["side"], case["reach"])
        st["rows"] = torch.tensor(_buckets(case["qh"], case["kh"], case["oy"], *rule), dtype=torch.int32, device=dev)
        st["cols"] = torch.tensor(_buckets(case["qw"], case["kw"], case["ox"], *rule), dtype=torch.int32, device=dev)
        if op == "bias":
            st["table"] = 0.5 * normal(s, s, heads)
            st["scores"] = None
            if case["scores"]:
                v = 2.0 * normal(n, heads, lq, lk)
                # some keys are padding, and so is all that some of the batch sees
                v.masked_fill_(torch.rand((n, 1, 1, lk), device=dev, generator=gen) < 0.05, -math.inf)
                v.masked_fill_(torch.rand((n, 1, 1, 1), device=dev, generator=gen) < 0.02, -math.inf)
                st["scores"] = v.to(dt)
            st["out"] = torch.empty((n, heads, lq, lk), dtype=dt, device=dev)
        else:
            st["dout"] = torch.empty((n, heads, lq, lk), dtype=dt, device=dev)
            for k in range(n):
                st["dout"][k] = normal(heads, lq, lk)
            st["dtable"] = torch.empty((s, s, heads), device=dev)
    return st


# ----------------------------------------------------------- the plain form

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
    return _phi(z) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_linear(st):
    c = st["case"]
    y = _act(st["x"].float() @ st["weight"].float().t() + st["bias"], c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"y": y.to(st["dtype"])}


def _plain_linear_grad(st):
    c = st["case"]
    dz = st["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(st["pre"].float(), c["act"])
    dx = (dz @ st["weight"].float()).to(st["dtype"])
    dz = dz.view(-1, c["k"])
    dweight = dz.t() @ st["x"].float().view(-1, c["c"])
    return {"dx": dx, "dweight": dweight.to(st["dtype"]), "dbias": dz.double().sum(0).float()}


def _angles(st):
    """Cosine and sine of every token's angles, (tokens, 1, pairs): row pairs, column pairs, pairs that stay."""
    c, dev = st["case"], st["x"].device
    n, h, w, f = c["n"], c["h"], c["w"], torch.float64
    if st["positions"] is None:
        py = torch.arange(h, device=dev, dtype=f).view(1, h, 1).expand(n, h, w).reshape(-1, 1)
        px = torch.arange(w, device=dev, dtype=f).view(1, 1, w).expand(n, h, w).reshape(-1, 1)
    else:
        py, px = st["positions"].to(f).view(-1, 2).split(1, 1)

    def turn(p, pairs):
        return p * c["base"] ** (-torch.arange(pairs, device=dev, dtype=f) / max(pairs, 1))

    a = torch.zeros((n * h * w, c["d"] // 2), device=dev, dtype=f)
    a[:, :c["row_pairs"]] = turn(py, c["row_pairs"])
    a[:, c["row_pairs"]:c["row_pairs"] + c["col_pairs"]] = turn(px, c["col_pairs"])
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _turned(v, cos, sin, interleaved):
    """v (tokens, heads, d) with its pairs turned."""
    out = torch.empty_like(v)
    if interleaved:
        a, b = v[..., 0::2], v[..., 1::2]
        out[..., 0::2], out[..., 1::2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = v.chunk(2, -1)
        half = v.shape[-1] // 2
        out[..., :half], out[..., half:] = a * cos - b * sin, a * sin + b * cos
    return out


def _heads(st, t):
    c = st["case"]
    heads = c["q_heads"] + c["k_heads"]
    return t[..., :heads * c["d"]].reshape(-1, heads, c["d"]).float()


def _plain_qk(st):
    c = st["case"]
    v = _heads(st, st["x"])
    u = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    u[:, :c["q_heads"]] *= st["gamma_q"]
    u[:, c["q_heads"]:] *= st["gamma_k"]
    return {"y": _turned(u, *_angles(st), c["interleaved"]).to(st["dtype"]).view(st["y"].shape)}


def _plain_qk_grad(st):
    c = st["case"]
    v, q = _heads(st, st["x"]), c["q_heads"]
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    xh = v * rstd
    cos, sin = _angles(st)
    du = _turned(_heads(st, st["dy"]), cos, -sin, c["interleaved"])
    t = du * xh
    dgq, dgk = t[:, :q].sum((0, 1)), t[:, q:].sum((0, 1))
    du[:, :q] *= st["gamma_q"]
    du[:, q:] *= st["gamma_k"]
    dx = rstd * (du - xh * (du * xh).mean(-1, keepdim=True))
    full = torch.zeros_like(st["x"])
    full[..., :dx.shape[1] * c["d"]] = dx.to(st["dtype"]).view(c["n"], c["h"], c["w"], -1)
    return {"dx": full, "dgamma_q": dgq, "dgamma_k": dgk}


def _pairs(st):
    """Bucket of every query and key, (queries, keys), in the table's order."""
    c, dev = st["case"], st["rows"].device

    def axis(buckets, queries, keys):
        q, k = torch.arange(queries, device=dev), torch.arange(keys, device=dev)
        return buckets.long()[k[None, :] - q[:, None] + queries - 1]

    r, x = axis(st["rows"], c["qh"], c["kh"]), axis(st["cols"], c["qw"], c["kw"])
    idx = r[:, None, :, None] * (2 * c["side"] - 1) + x[None, :, None, :]
    return idx.reshape(c["qh"] * c["qw"], c["kh"] * c["kw"])


def _plain_bias(st):
    c = st["case"]
    b = st["table"].view(-1, c["heads"])[_pairs(st)].permute(2, 0, 1)
    if st["scores"] is None:
        return {"out": b.to(st["dtype"]).expand(c["n"], -1, -1, -1).contiguous()}
    return {"out": (st["scores"].float() + b).to(st["dtype"])}


def _plain_bias_grad(st):
    c = st["case"]
    s = 2 * c["side"] - 1
    d = st["dout"].sum(0, dtype=torch.float64).view(c["heads"], -1)
    out = torch.zeros((c["heads"], s * s), dtype=torch.float64, device=d.device)
    out.index_add_(1, _pairs(st).view(-1), d)
    return {"dtable": out.t().reshape(s, s, c["heads"]).float()}


_PLAIN = {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "qk_norm": _plain_qk,
          "qk_norm_grad": _plain_qk_grad, "bias": _plain_bias, "bias_grad": _plain_bias_grad}


# ------------------------------------------------------ the framework's calls

def _own(st):
    import bilinear_image_resize_gb300 as rz
    c = st["case"]
    if c["op"] in ("linear", "linear_grad"):
        act = {"none": rz.RZ_ACT_NONE, "silu": rz.RZ_ACT_SILU, "gelu": rz.RZ_ACT_GELU}[c["act"]]
    if c["op"] == "linear":
        rz.map_linear(st["x"], st["y"], st["weight"], st["bias"], residual=st["residual"], act=act)
        return {"y": st["y"]}
    if c["op"] == "linear_grad":
        rz.map_linear_grad(st["dy"], st["x"], st["weight"], st["dx"], st["dweight"], st["dbias"], pre=st["pre"], act=act)
        return {"dx": st["dx"], "dweight": st["dweight"], "dbias": st["dbias"]}
    if c["op"] in ("qk_norm", "qk_norm_grad"):
        turn = dict(base=c["base"], row_pairs=c["row_pairs"], col_pairs=c["col_pairs"], interleaved=c["interleaved"],
                    positions=st["positions"], eps=EPS)
    if c["op"] == "qk_norm":
        rz.map_qk_norm(st["x"], st["y"], c["q_heads"], c["k_heads"], c["d"], st["gamma_q"], st["gamma_k"], **turn)
        return {"y": st["y"]}
    if c["op"] == "qk_norm_grad":
        rz.map_qk_norm_grad(st["dy"], st["x"], st["dx"], c["q_heads"], c["k_heads"], c["d"], st["gamma_q"],
                            st["gamma_k"], st["dgamma_q"], st["dgamma_k"], **turn)
        return {"dx": st["dx"], "dgamma_q": st["dgamma_q"], "dgamma_k": st["dgamma_k"]}
    grids = ((c["qh"], c["qw"]), (c["kh"], c["kw"]))
    if c["op"] == "bias":
        rz.map_position_bias(st["table"], st["rows"], st["cols"], st["out"], *grids, scores=st["scores"])
        return {"out": st["out"]}
    rz.map_position_bias_grad(st["dout"], st["rows"], st["cols"], st["dtable"], *grids)
    return {"dtable": st["dtable"]}


def run(st):
    return _own(st) if own else _PLAIN[st["case"]["op"]](st)


# -------------------------------------------------------- the same in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op, f, dev = case["op"], torch.float64, "cuda"

    def slopes(z):
        """The activation and its derivative."""
        if case["act"] == "silu":
            s = torch.sigmoid(z)
            return z * s, s + z * s * (1 - s)
        if case["act"] == "gelu":
            s = torch.special.ndtr(z)
            return z * s, s + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z, torch.ones_like(z)

    if op in ("linear", "linear_grad"):
        w = st["weight"].to(f)
        if op == "linear":
            y = torch.empty(st["y"].shape, dtype=f, device=dev)
            for k in range(case["n"]):
                y[k] = slopes(torch.einsum("hwc,kc->hwk", st["x"][k].to(f), w) + st["bias"].to(f))[0]
            return {"y": y if st["residual"] is None else y.add_(st["residual"].to(f))}
        dx, dw = torch.empty(st["dx"].shape, dtype=f, device=dev), torch.zeros_like(w)
        db = torch.zeros(case["k"], dtype=f, device=dev)
        for k in range(case["n"]):
            dz = st["dy"][k].to(f)
            if st["pre"] is not None:
                dz = dz * slopes(st["pre"][k].to(f))[1]
            dx[k] = torch.einsum("hwk,kc->hwc", dz, w)
            dw += torch.einsum("hwk,hwc->kc", dz, st["x"][k].to(f))
            db += dz.sum((0, 1))
        return {"dx": dx, "dweight": dw, "dbias": db}

    if op in ("qk_norm", "qk_norm_grad"):
        n, h, w, d, q, k = (case[i] for i in ("n", "h", "w", "d", "q_heads", "k_heads"))
        z = torch.zeros((n, h, w, 2), dtype=f, device=dev)
        if st["positions"] is None:
            z[..., 0] += torch.arange(h, dtype=f, device=dev)[:, None]
            z[..., 1] += torch.arange(w, dtype=f, device=dev)
        else:
            z += st["positions"]
        spin = torch.ones((n, h, w, 1, d // 2), dtype=torch.complex128, device=dev)
        at = 0
        for axis, pairs in ((0, case["row_pairs"]), (1, case["col_pairs"])):
            for j in range(pairs):
                a = z[..., axis] / case["base"] ** (j / pairs)
                spin[..., 0, at] = torch.polar(torch.ones_like(a), a)
                at += 1

        def spun(v, by):
            v = v.view(n, h, w, q + k, d)
            p = v.unflatten(-1, (d // 2, 2)) if case["interleaved"] else v.unflatten(-1, (2, d // 2)).transpose(-1, -2)
            p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * by)
            return (p if case["interleaved"] else p.transpose(-1, -2)).flatten(-2)

        x = st["x"][..., :(q + k) * d].to(f).reshape(n, h, w, q + k, d)
        r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        gamma = torch.cat([st["gamma_q"].to(f).expand(q, d), st["gamma_k"].to(f).expand(k, d)])
        if op == "qk_norm":
            return {"y": spun(x * r * gamma, spin).reshape(st["y"].shape)}
        du = spun(st["dy"].to(f), spin.conj())
        dg = torch.einsum("nhwgd,nhwgd->gd", du, x * r)
        du = du * gamma
        dx = torch.zeros(st["x"].shape, dtype=f, device=dev)
        dx[..., :(q + k) * d] = (r * du - x * r ** 3 * ((du * x).sum(-1, keepdim=True) / d)).reshape(n, h, w, -1)
        return {"dx": dx, "dgamma_q": dg[:q].sum(0), "dgamma_k": dg[q:].sum(0)}

    s, heads = 2 * case["side"] - 1, case["heads"]
    qh, qw, kh, kw = (case[i] for i in ("qh", "qw", "kh", "kw"))

    def members(buckets, queries, keys):
        """(queries, keys, buckets): 1 where a pair is of the bucket."""
        m = torch.zeros((queries, keys, s), dtype=f, device=dev)
        b = buckets.tolist()
        for i in range(queries):
            m[i, torch.arange(keys), b[queries - 1 - i:queries - 1 - i + keys]] = 1
        return m

    r, c = members(st["rows"], qh, kh), members(st["cols"], qw, kw)
    if op == "bias":
        out = torch.empty(st["out"].shape, dtype=f, device=dev)
        for a in range(heads):
            half = torch.einsum("yur,rc->yuc", r, st["table"][..., a].to(f))
            b = torch.einsum("yuc,xvc->yxuv", half, c).reshape(qh * qw, kh * kw)
            out[:, a] = b if st["scores"] is None else st["scores"][:, a].to(f) + b
        return {"out": out}
    out = torch.zeros((s, s, heads), dtype=f, device=dev)
    for a in range(heads):
        d = torch.zeros((qh * qw, kh * kw), dtype=f, device=dev)
        for k in range(case["n"]):
            d += st["dout"][k, a]
        half = torch.einsum("yxuv,xvc->yuc", d.view(qh, qw, kh, kw), c)
        out[..., a] = torch.einsum("yuc,yur->rc", half, r)
    return {"dtable": out}

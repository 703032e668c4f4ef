"""Cases that time the appearance operators: the shared feature table, the shading network's
normalisation and the orthogonalised update.

`run` computes a case in elementary torch operations in 32 bits where `own` is false, and through
sphere_rasterization_amd.appearance where it is true. `exact` computes the same from the
definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
NORM_EPS = 1e-5
ORTHO_EPS = 1e-7
MOST = 2_000_000 * 64          # values of the largest array of a case


def _lookup(op, n, rows, dim, dtype, ids, skew, scale, name=None):
    c = dict(op=op, n=n, rows=rows, dim=dim, dtype=dtype, ids=ids, skew=skew, scale=scale)
    return dict(c, name=name) if name else c


def _norm(op, images, height, width, channels, groups, dtype, act, name=None):
    c = dict(op=op, images=images, height=height, width=width, channels=channels, groups=groups, dtype=dtype, act=act)
    return dict(c, name=name) if name else c


def _ortho(batch, rows, cols, dtype, name=None):
    c = dict(op="orthogonalize", batch=batch, rows=rows, cols=cols, dtype=dtype)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one id, as when a single entry is fetched between frames: latency alone
        _lookup("lookup", 1, 65536, 64, "f32", "int64", False, 1.0, "lookup_one"),
        # the features of the 2M-primitive driving scene, 32 channels, from one table
        _lookup("lookup", 2_000_000, 65536, 32, "f32", "int32", True, 0.5, "lookup_driving"),
        # the 4,096 primitives of the smallest scene, 3 channels, a palette of 256
        _lookup("lookup_grad", 4096, 256, 3, "f32", "int32", False, 1.0, "grad_tiny"),
        # the driving scene's table gradient, few entries holding most primitives
        _lookup("lookup_grad", 2_000_000, 65536, 32, "f32", "int32", True, 0.5, "grad_driving"),
        # wide rows, as in a text encoder's vocabulary next to the scene: an odd number of tokens and of rows
        _lookup("lookup_grad", 16383, 50001, 2048, "bf16", "int64", True, 45.25, "grad_tokens"),
        # one ragged patch of a feature image shaded on its own
        _norm("norm", 1, 33, 47, 64, 8, "bf16", "silu", "norm_patch"),
        # a full 1920x1080 feature image of 32 channels shaded for display
        _norm("norm", 1, 1080, 1920, 32, 8, "f16", "silu", "norm_1080p"),
        # training on the 1024x1024 sphere frame, forward and backward
        _norm("norm_grad", 1, 1024, 1024, 32, 8, "f32", "silu", "train_norm_spheres"),
        # training on the six 1280x720 cameras of the rig, 24 channels
        _norm("norm_grad", 6, 720, 1280, 24, 4, "bf16", "gelu", "train_norm_rig"),
        # the update of a small shading network: eight 64x32 matrices at once
        _ortho(8, 64, 32, "f32", "ortho_shader"),
        # one odd-sized matrix, taller than wide
        _ortho(1, 1000, 777, "bf16", "ortho_odd"),
        # one large matrix
        _ortho(1, 2048, 4096, "f32", "ortho_large"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["lookup", "lookup_grad", "norm", "norm_grad", "orthogonalize"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind in ("lookup", "lookup_grad"):
        if rng.random() < 0.7:     # primitives: few channels, many of them
            dim, n, rows = rng.randint(1, 64), _log(rng, 1, 2_000_000), _log(rng, 1, 200_000)
        else:                      # wide rows
            dim = _log(rng, 65, 4096)
            n, rows = _log(rng, 1, min(65536, MOST // dim)), _log(rng, 16, min(100_000, MOST // dim))
        return _lookup(kind, n, rows, dim, dtype, rng.choice(["int32", "int64"]), rng.random() < 0.5,
                       rng.choice([1.0, 0.5, 8.0]))
    if kind in ("norm", "norm_grad"):
        groups = rng.choice([1, 2, 4, 8, 16, 32])
        channels = groups * rng.choice([1, 2, 3, 4, 6, 8, 16])
        images = rng.randint(1, 6)
        most = min(1920 * 1080, MOST // (channels * images))
        pixels = _log(rng, 4, most)
        width = max(1, min(pixels, int(math.sqrt(pixels) * rng.uniform(0.7, 1.9))))
        # relu's slope jumps at 0, where no two roundings agree on the side: forward only
        return _norm(kind, images, max(1, pixels // width), width, channels, groups, dtype,
                     rng.choice(["none", "silu", "gelu"] + (["relu"] if kind == "norm" else [])))
    batch = rng.choice([1, 1, 2, 4, 8])
    rows, cols = _log(rng, 8, 2048), _log(rng, 8, 2048)
    return _ortho(batch, rows, cols, dtype)


def _ids(case, gen):
    n, rows = case["n"], case["rows"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case["skew"]:               # a few entries hold most tokens: id ~ rows^u, log-uniform
        v = torch.exp(u * math.log(rows + 1.0)) - 1.0
    else:
        v = u * rows
    ids = v.long().clamp_(0, rows - 1)
    if n > 1:                      # one in a hundred has no entry
        ids[torch.rand(n, generator=gen, device="cuda") < 0.01] = -1
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "lookup":
        s["table"] = _randn(gen, case["rows"], case["dim"]).to(dt)
        s["ids"] = _ids(case, gen)
    elif case["op"] == "lookup_grad":
        s["dy"] = _randn(gen, case["n"], case["dim"]).to(dt)
        s["ids"] = _ids(case, gen)
    elif case["op"] in ("norm", "norm_grad"):
        shape = (case["images"], case["height"], case["width"], case["channels"])
        c = case["channels"]
        s["x"] = (_randn(gen, *shape) * (0.5 + torch.rand(c, generator=gen, device="cuda")) + _randn(gen, c)).to(dt)
        s["weight"] = (1.0 + 0.2 * _randn(gen, c)).to(dt)
        s["bias"] = (0.2 * _randn(gen, c)).to(dt)
        if case["op"] == "norm_grad":
            s["dy"] = _randn(gen, *shape).to(dt)
    else:
        b, r, c = case["batch"], case["rows"], case["cols"]
        k = max(1, min(r, c) // 8)     # a momentum: a few strong directions over noise
        g = torch.bmm(_randn(gen, b, r, k), _randn(gen, b, k, c)) * (2.0 / math.sqrt(k)) + _randn(gen, b, r, c)
        s["g"] = (1e-3 * g).to(dt)
    return s


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "silu":
        t = 1.0 / (1.0 + torch.exp(-z))
        return t * (1.0 + z * (1.0 - t))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain_norm(s, wide):
    """Outputs of a norm case in the type `wide`, before the last rounding."""
    case = s["case"]
    n, c, g = case["images"], case["channels"], case["groups"]
    x = s["x"].to(wide).view(n, -1, g, c // g)
    w, b = s["weight"].to(wide).view(g, c // g), s["bias"].to(wide).view(g, c // g)
    mean = x.mean(dim=(1, 3), keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=(1, 3), keepdim=True) + NORM_EPS)
    xh = xc * rstd
    z = xh * w + b
    y = _act(z, case["act"]).view(s["x"].shape)
    if case["op"] == "norm":
        return (y,)
    dz = s["dy"].to(wide).view(n, -1, g, c // g) * _act_slope(z, case["act"])
    dzx = dz * xh
    db, dw = dz.sum(dim=(0, 1)).view(c), dzx.sum(dim=(0, 1)).view(c)
    s1 = (dz * w).mean(dim=(1, 3), keepdim=True)
    s2 = (dzx * w).mean(dim=(1, 3), keepdim=True)
    dx = (dz * w - s1 - xh * s2) * rstd
    return y, dx.view(s["x"].shape), dw, db


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "lookup":
        ids, table = s["ids"].long(), s["table"]
        none = (ids < 0) | (ids >= case["rows"])
        y = table[ids.clamp(0, case["rows"] - 1)].float() * case["scale"]
        return y.masked_fill_(none[:, None], 0.0).to(dt)
    if case["op"] == "lookup_grad":
        ids = s["ids"].long()
        at = torch.where((ids < 0) | (ids >= case["rows"]), case["rows"], ids)
        d = torch.zeros(case["rows"] + 1, case["dim"], device="cuda")
        return (d.index_add_(0, at, s["dy"].float())[:case["rows"]] * case["scale"]).to(dt)
    if case["op"] in ("norm", "norm_grad"):
        return tuple(v.to(dt) for v in _plain_norm(s, torch.float32))
    x = s["g"].float()
    tall = case["rows"] > case["cols"]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (torch.sqrt((x * x).sum(dim=(1, 2), keepdim=True)) + ORTHO_EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return (x.transpose(1, 2).contiguous() if tall else x).to(dt)


def _call(s):
    from sphere_rasterization_amd import appearance as A
    case = s["case"]
    if case["op"] == "lookup":
        return A.lookup(s["table"], s["ids"], scale=case["scale"])
    if case["op"] == "lookup_grad":
        return A.lookup_backward(s["dy"], s["ids"], case["rows"], scale=case["scale"])
    if case["op"] == "norm":
        return (A.group_norm(s["x"], case["groups"], s["weight"], s["bias"], eps=NORM_EPS, act=case["act"]),)
    if case["op"] == "norm_grad":
        y, mean, rstd = A.group_norm_forward(s["x"], case["groups"], s["weight"], s["bias"], eps=NORM_EPS,
                                             act=case["act"])
        dx, dw, db = A.group_norm_backward(s["dy"], s["x"], mean, rstd, s["weight"], s["bias"], act=case["act"])
        return y, dx, dw, db
    return A.orthogonalize(s["g"], steps=STEPS, coeffs=COEFFS, eps=ORTHO_EPS)


def run(state):
    return _call(state) if own else _plain(state)


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"] in ("lookup", "lookup_grad"):
        n, rows, dim = case["n"], case["rows"], case["dim"]
        ids = n * (4 if case["ids"] == "int32" else 8)
        table = (min(n, rows) if case["op"] == "lookup" else rows) * dim * e
        return {"bytes": ids + n * dim * e + table, "flops": n * dim}
    if case["op"] in ("norm", "norm_grad"):
        v = case["images"] * case["height"] * case["width"] * case["channels"]
        p = case["channels"] * e
        if case["op"] == "norm":
            return {"bytes": 2 * v * e + 2 * p, "flops": 8 * v}
        return {"bytes": 4 * v * e + 4 * p, "flops": 24 * v}
    m, n = sorted((case["rows"], case["cols"]))
    # per step: half of the symmetric X X^T and A A, and all of B X
    flops = case["batch"] * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    return {"bytes": 2 * case["batch"] * m * n * e, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lookup":
        ids, dim = s["ids"].long(), case["dim"]
        ok = (ids >= 0) & (ids < case["rows"])
        y = torch.zeros(case["n"], dim, device="cuda", dtype=torch.float64)
        y[ok] = s["table"].double()[ids[ok]] * case["scale"]
        return y
    if case["op"] == "lookup_grad":
        ids = s["ids"].long()
        ok = (ids >= 0) & (ids < case["rows"])
        d = torch.zeros(case["rows"], case["dim"], device="cuda", dtype=torch.float64)
        d.index_put_((ids[ok],), s["dy"].double()[ok] * case["scale"], accumulate=True)
        return d
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(s)
    return _exact_ortho(s["g"])


def _exact_norm(s):
    """Group by group, from the definition; the gradient through the centred values."""
    case = s["case"]
    n, c, g = case["images"], case["channels"], case["groups"]
    k = c // g
    out = [torch.empty(s["x"].shape, device="cuda", dtype=torch.float64)]
    train = case["op"] == "norm_grad"
    if train:
        out += [torch.empty_like(out[0])] + [torch.zeros(c, device="cuda", dtype=torch.float64) for _ in range(2)]
    for i in range(n):
        for j in range(g):
            at = slice(j * k, j * k + k)
            x = s["x"][i, ..., at].double()
            w, b = s["weight"][at].double(), s["bias"][at].double()
            var, mean = torch.var_mean(x, correction=0)
            sd = torch.sqrt(var + NORM_EPS)
            h = (x - mean) / sd
            z = w * h + b
            out[0][i, ..., at] = _act(z, case["act"])
            if train:
                d = s["dy"][i, ..., at].double() * _act_slope(z, case["act"])
                out[2][at] += (d * h).sum(dim=(0, 1))
                out[3][at] += d.sum(dim=(0, 1))
                dh = d * w
                out[1][i, ..., at] = (dh - dh.mean() - h * (dh * h).mean()) / sd
    return tuple(out)


def _exact_ortho(g):
    """The same polynomial applied to the singular values."""
    if g.shape[1] * g.shape[2] > 1024 * 1024:
        return _exact_ortho_products(g)
    u, sv, vt = torch.linalg.svd(g.double().cpu(), full_matrices=False)
    sv = sv / (torch.sqrt((sv * sv).sum(dim=1, keepdim=True)) + ORTHO_EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        sv = a * sv + b * sv ** 3 + c * sv ** 5
    return torch.matmul(u * sv[:, None, :], vt).cuda()


def _exact_ortho_products(g):
    """Matrices too large for their singular values in time: the products, in 64 bits."""
    x = g.double()
    if x.shape[1] > x.shape[2]:
        return _exact_ortho_products(g.transpose(1, 2).contiguous()).transpose(1, 2).contiguous()
    x = x / (torch.linalg.matrix_norm(x)[:, None, None] + ORTHO_EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        gram = torch.matmul(x, x.transpose(1, 2).contiguous())
        x3 = torch.matmul(gram, x)
        x = a * x + b * x3 + c * torch.matmul(gram, x3)
    return x

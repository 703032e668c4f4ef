"""Cases that time the dense layers of a shading network: the product with bias, activation, dropout
and residual in its epilogue, its gradient, and dropout on its own.

    y = residual + keep * act(x W + b) / (1 - p)

`run` computes a case in elementary torch operations in 32 bits where `own` is false, and through
sphere_rasterization_amd.appearance where it is true. `exact` computes the same from the
definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
MOST = 2_073_600 * 64              # values of the largest array of a case
MOST_WIDE = 8191 * 1024 * 4096     # multiply-adds of the largest product


def _linear(op, rows, k, n, dtype, act, bias, residual, p, order, name=None):
    """order "io": W is stored [in][out]; "oi": [out][in], handed over as its transpose."""
    c = dict(op=op, rows=rows, k=k, n=n, dtype=dtype, act=act, bias=bias, residual=residual, p=p, order=order)
    return dict(c, name=name) if name else c


def _dropout(op, rows, n, dtype, residual, p, state, name=None):
    """state: seed and offset lie on the GPU, as for a step that is captured and replayed."""
    c = dict(op=op, rows=rows, n=n, dtype=dtype, residual=residual, p=p, state=state)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the colour of one primitive picked in the viewer: latency alone
        _linear("linear", 1, 64, 32, "f32", "silu", True, False, 0.0, "io", "linear_one"),
        # one token of a text encoder next to the scene: its weights are read for a single row
        _linear("linear", 1, 2048, 8192, "bf16", "gelu", True, False, 0.0, "oi", "linear_token"),
        # the hidden layer over a full 1920x1080 feature image of 32 channels, for display
        _linear("linear", 2_073_600, 32, 64, "f16", "silu", True, False, 0.0, "io", "linear_1080p"),
        # tokens of the encoder through its widening layer
        _linear("linear", 8191, 1024, 4096, "bf16", "gelu", True, False, 0.0, "io", "linear_wide"),
        # a deep per-image layer in full precision, with the residual that skips it
        _linear("linear", 4095, 1536, 1000, "f32", "none", True, True, 0.0, "oi", "linear_f32"),
        # one ragged patch of a feature image, trained with dropout
        _linear("linear_grad", 33 * 47, 65, 130, "f16", "silu", True, True, 0.1, "io", "train_patch"),
        # training on the 1024x1024 sphere frame of 32 channels
        _linear("linear_grad", 1024 * 1024, 32, 32, "f32", "silu", True, True, 0.0, "io", "train_spheres"),
        # training on the six 1280x720 cameras of the rig, 24 channels to 32, with dropout
        _linear("linear_grad", 6 * 720 * 1280, 24, 32, "bf16", "gelu", True, False, 0.1, "io", "train_rig"),
        # training the widening layer, with dropout
        _linear("linear_grad", 8191, 1024, 4096, "bf16", "gelu", True, False, 0.1, "io", "train_wide"),
        # dropout of one patch's features: latency alone
        _dropout("dropout", 33 * 47, 64, "bf16", False, 0.1, False, "dropout_patch"),
        # a full 1920x1080 image of 32 channels dropped and added to its residual
        _dropout("dropout", 2_073_600, 32, "f16", True, 0.25, True, "dropout_1080p"),
        # colours of an odd number of pixels, forward and backward
        _dropout("dropout_grad", 1023 * 1021, 3, "f32", False, 0.5, False, "dropout_grad_rgb"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear_grad", "linear_grad", "dropout", "dropout_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    residual = rng.random() < 0.4
    if kind in ("dropout", "dropout_grad"):
        n = _log(rng, 1, 4096)
        return _dropout(kind, _log(rng, 1, MOST // 2 // n), n, dtype, residual, rng.choice([0.1, 0.25, 0.5, 0.9]),
                        rng.random() < 0.5)
    shape = rng.random()
    if shape < 0.5:                # pixels or primitives: few channels, many of them
        k, n = rng.randint(1, 64), rng.randint(1, 64)
        rows = _log(rng, 1, 2_073_600)
    elif shape < 0.75:             # wide rows
        k, n = _log(rng, 65, 4096), _log(rng, 65, 4096)
        rows = _log(rng, 17, min(16384, MOST_WIDE // (k * n)))
    else:                          # wide rows, one to a few of them
        k, n = _log(rng, 65, 8192), _log(rng, 65, 8192)
        rows = rng.randint(1, 16)
    # relu's slope jumps at 0, where no two roundings agree on the side: forward only
    act = rng.choice(["none", "silu", "gelu"] + (["relu"] if kind == "linear" else []))
    p = rng.choice([0.0, 0.1, 0.5]) if kind == "linear_grad" else 0.0
    return _linear(kind, rows, k, n, dtype, act, rng.random() < 0.7, residual, p, rng.choice(["io", "oi"]))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    rows, n = case["rows"], case["n"]
    # what a training loop draws from: its seed, and a number of its own for every step and layer
    s = dict(case=case, seed=0x9E3779B97F4A7C15 ^ seed, offset=(1 << 33) + seed)
    if case["op"] in ("linear", "linear_grad"):
        k = case["k"]
        s["x"] = _randn(gen, rows, k).mul_(0.5 + torch.rand(k, generator=gen, device="cuda")).to(dt)
        if case["order"] == "io":
            s["w"] = (_randn(gen, k, n) * k ** -0.5).to(dt)
        else:
            s["w"] = (_randn(gen, n, k) * k ** -0.5).to(dt).t()
        s["bias"] = (0.2 * _randn(gen, n)).to(dt) if case["bias"] else None
    else:
        s["x"] = _randn(gen, rows, n).to(dt)
        if case["state"]:
            words = [v - (1 << 64) if v >= 1 << 63 else v for v in (s["seed"], s["offset"])]
            s["state"] = torch.tensor(words, dtype=torch.int64, device="cuda")
    s["residual"] = _randn(gen, rows, n).to(dt) if case["residual"] else None
    if case["op"] in ("linear_grad", "dropout_grad"):
        s["dy"] = _randn(gen, rows, n).to(dt)
    return s


# ---- the plain form ------------------------------------------------------------------

def _philox(block, half, seed, offset):
    """The four words of Philox4x32-10 for int64 tensors of block numbers, as int64."""
    low = 0xFFFFFFFF

    def product(a, m):             # high and low word of a * m: a * m itself does not fit 63 bits
        high = ((a >> 16) * m + (((a & 0xFFFF) * m) >> 16)) >> 16
        return high, (a * m) & low

    c = [block & low, (block >> 32) | (half << 31), torch.full_like(block, offset & low), torch.full_like(block, offset >> 32)]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c


def _factor(s, shape):
    """What dropout multiplies each element by, in 32 bits: 0 or 1 / (1 - p)."""
    p = s["case"]["p"]
    n = math.prod(shape)
    block = torch.arange((n + 7) // 8, device="cuda")
    pieces = []
    for half in (0, 1):            # the upper and the lower 16 bits of each element's number
        words = torch.stack(_philox(block, half, s["seed"], s["offset"]), dim=1)
        pieces.append(torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(-1)[:n])
    u = (pieces[0] << 16) | pieces[1]
    scale = 1.0 / (1.0 - p) if p < 1.0 else 0.0
    return (u >= round(p * 2.0 ** 32)).float().mul_(scale).view(shape)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    return z


def _act_slope(z, act):
    if act == "silu":
        t = 1.0 / (1.0 + torch.exp(-z))
        return t * (1.0 + z * (1.0 - t))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    shape = (case["rows"], case["n"])
    res = s["residual"]
    if case["op"] in ("dropout", "dropout_grad"):
        f = _factor(s, shape)
        y = s["x"].float() * f
        y = (y if res is None else y + res.float()).to(dt)
        return y if case["op"] == "dropout" else (y, (s["dy"].float() * f).to(dt))
    x, w = s["x"].float(), s["w"].float()
    z = torch.matmul(x, w)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, case["act"])
    f = _factor(s, shape) if case["p"] > 0 else None
    if f is not None:
        y = y * f
    if res is not None:
        y = y + res.float()
    y = y.to(dt)
    if case["op"] == "linear":
        return y
    dz = s["dy"].float()
    if f is not None:
        dz = dz * f
    if case["act"] != "none":
        dz = dz * _act_slope(z, case["act"])
    dx, dw = torch.matmul(dz, w.t()), torch.matmul(x.t(), dz)
    db = dz.sum(dim=0).to(dt) if s["bias"] is not None else None
    return {k: v for k, v in dict(y=y, dx=dx.to(dt), dw=dw.to(dt), db=db).items() if v is not None}


# ---- the framework's calls -----------------------------------------------------------

def _call(s):
    from sphere_rasterization_amd import appearance as A
    case = s["case"]
    if case["op"] in ("dropout", "dropout_grad"):
        rng = (s["state"], 0) if case["state"] else (s["seed"], s["offset"])
        y = A.dropout(s["x"], case["p"], rng, residual=s["residual"])
        return y if case["op"] == "dropout" else (y, A.dropout_backward(s["dy"], case["p"], rng))
    rng = (s["seed"], s["offset"]) if case["p"] > 0 else None
    more = dict(act=case["act"], p=case["p"], rng=rng)
    if case["op"] == "linear":
        return A.linear(s["x"], s["w"], s["bias"], residual=s["residual"], **more)
    y, pre = A.linear_forward(s["x"], s["w"], s["bias"], residual=s["residual"], **more)
    want = ("x", "weight", "bias") if case["bias"] else ("x", "weight")
    dx, dw, db = A.linear_backward(s["dy"], s["x"], s["w"], s["bias"], pre=pre, want=want, **more)
    return {k: v for k, v in dict(y=y, dx=dx, dw=dw, db=db).items() if v is not None}


def run(state):
    return _call(state) if own else _plain(state)


def work(case):
    e, rows, n = SIZES[case["dtype"]], case["rows"], case["n"]
    out = rows * n
    if case["op"] in ("dropout", "dropout_grad"):
        arrays = 2 + (1 if case["residual"] else 0) + (2 if case["op"] == "dropout_grad" else 0)
        return {"bytes": arrays * out * e, "flops": 2 * out}
    k = case["k"]
    weights = k * n + (n if case["bias"] else 0)
    arrays = rows * k + weights + out + (out if case["residual"] else 0)
    if case["op"] == "linear":
        return {"bytes": arrays * e, "flops": 2 * rows * n * k}
    # the backward reads dy, x and the weights and writes as much as x and the weights hold
    return {"bytes": (arrays + out + 2 * rows * k + 2 * weights) * e, "flops": 6 * rows * n * k}


# ---- the definition in 64 bits -------------------------------------------------------

def _words(block, half, seed, offset):
    """Philox4x32-10 by numpy's unsigned 64-bit products."""
    u, mask, by = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    x0, x1 = block & mask, (block >> by) | u(half << 31)
    x2, x3 = np.full_like(block, offset & 0xFFFFFFFF), np.full_like(block, offset >> 32)
    for r in range(10):
        key0 = u((seed + r * 0x9E3779B9) & 0xFFFFFFFF)
        key1 = u(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        a, b = x0 * u(0xD2511F53), x2 * u(0xCD9E8D57)
        x0, x1, x2, x3 = (b >> by) ^ x1 ^ key0, b & mask, (a >> by) ^ x3 ^ key1, a & mask
    return x0, x1, x2, x3


def _pieces(block, half, seed, offset):
    """[blocks, 8]: the eight 16-bit pieces of each block, low half of each word first."""
    w = np.stack([v.astype("<u4") for v in _words(block, half, seed, offset)], axis=1)
    return w.view("<u2").astype(np.int64)


def _kept(s, shape):
    """Truth values: which elements dropout keeps. The second draw is made where the first ties."""
    p, n = s["case"]["p"], math.prod(shape)
    t = round(p * 2.0 ** 32)
    keep = np.empty(((n + 7) // 8, 8), dtype=bool)
    for at in range(0, keep.shape[0], 1 << 20):
        block = np.arange(at, min(at + (1 << 20), keep.shape[0]), dtype=np.uint64)
        hi = _pieces(block, 0, s["seed"], s["offset"])
        k = hi > t >> 16
        tie = np.nonzero((hi == t >> 16).any(axis=1))[0]
        if tie.size:
            lo = _pieces(block[tie], 1, s["seed"], s["offset"])
            k[tie] |= (hi[tie] == t >> 16) & (lo >= (t & 0xFFFF))
        keep[at:at + block.size] = k
    return torch.from_numpy(keep.reshape(-1)[:n].reshape(shape)).cuda()


def _slope64(z, act):
    if act == "silu":
        return torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z)
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return None


def _value64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def exact(case, seed):
    s = prepare(case, seed)
    p = case["p"]
    keep = _kept(s, (case["rows"], case["n"])) if p > 0 else None

    def dropped(v):
        return v if keep is None else torch.where(keep, v / (1.0 - p), torch.zeros_like(v))

    if case["op"] in ("dropout", "dropout_grad"):
        y = dropped(s["x"].double())
        if case["residual"]:
            y += s["residual"].double()
        return y if case["op"] == "dropout" else (y, dropped(s["dy"].double()))
    x, w = s["x"].double(), s["w"].double().contiguous()
    z = x @ w
    if case["bias"]:
        z += s["bias"].double()
    y = dropped(_value64(z, case["act"]))
    if case["residual"]:
        y += s["residual"].double()
    if case["op"] == "linear":
        return y
    d = dropped(s["dy"].double())
    slope = _slope64(z, case["act"])
    if slope is not None:
        d *= slope
    out = dict(y=y, dx=d @ w.t().contiguous(), dw=torch.zeros(case["k"], case["n"], device="cuda", dtype=torch.float64))
    for at in range(0, case["rows"], 1 << 18):
        out["dw"] += x[at:at + (1 << 18)].t().contiguous() @ d[at:at + (1 << 18)]
    if case["bias"]:
        out["db"] = d.sum(dim=0)
    return out

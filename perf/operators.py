"""Cases of the layer operators: the residual RMS norm, the distillation loss
from a teacher's top logits, and microscaled 4-bit matrices (quantisation and
product), each in the forms a training step calls them in.

A case names an operator ("op") and its sizes:

  norm     h = x + r, y = RMSnorm(h) w; out "16" (the input's type) or "e4m3"
           with one scale per row (block 0) or per 128 columns (block 128);
           train: the backward pass too (dx, dw)
  distill  the loss of each row against the teacher's k logits, and the
           gradient of the student's logits, scaled by the loss scale
  mx4      quantise a matrix along its rows (and, both: along its columns) to
           4 bits with a scale per 32, and the values back in its own type
  linear   y = x w^T with both operands in 4 bits; the weight is in hand in
           4 bits (train False), or 16-bit x, w and dy give y, dx and dw
           (train True)
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token of the GPT-2 shaped model: latency
        {"name": "norm 1x1600 f16", "op": "norm", "rows": 1, "cols": 1600, "dtype": "f16", "out": "16", "block": 0,
         "train": False},
        # a batch's activations of the Llama-3-8B shaped model, handed to an 8-bit product
        {"name": "norm 16384x4096 bf16 e4m3", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "out": "e4m3", "block": 128, "train": False},
        # one micro-batch's training pass of the same model
        {"name": "norm 8192x4096 bf16 train", "op": "norm", "rows": 8192, "cols": 4096, "dtype": "bf16", "out": "16",
         "block": 0, "train": True},
        # a ragged batch of an odd width: no row but the first on a 16-byte boundary
        {"name": "norm 2047x1337 f16 train", "op": "norm", "rows": 2047, "cols": 1337, "dtype": "f16", "out": "16",
         "block": 0, "train": True},
        # a few tokens against the GPT-2 vocabulary (odd: rows start anywhere)
        {"name": "distill 3x50257 f16 k8", "op": "distill", "rows": 3, "cols": 50257, "k": 8, "dtype": "f16",
         "temperature": 2.0, "scale": 1024.0},
        # a micro-batch against the Llama-3 vocabulary
        {"name": "distill 4096x128256 bf16 k64", "op": "distill", "rows": 4096, "cols": 128256, "k": 64,
         "dtype": "bf16", "temperature": 1.0, "scale": 1.0},
        # fp32 logits, a ragged batch
        {"name": "distill 1999x50257 f32 k33", "op": "distill", "rows": 1999, "cols": 50257, "k": 33, "dtype": "f32",
         "temperature": 2.0, "scale": 1.0},
        # the gate matrix of a Llama-3-8B shaped block, for the forward and the backward product
        {"name": "mx4 14336x4096 bf16 both", "op": "mx4", "rows": 14336, "cols": 4096, "dtype": "bf16", "both": True},
        # a ragged few rows in fp32
        {"name": "mx4 77x1600 f32 rows", "op": "mx4", "rows": 77, "cols": 1600, "dtype": "f32", "both": False},
        # one token through the gate matrix, the weight in 4 bits
        {"name": "linear 1x14336x4096 bf16", "op": "linear", "rows": 1, "n": 14336, "k": 4096, "dtype": "bf16",
         "train": False},
        # a micro-batch through the gate matrix
        {"name": "linear 8192x14336x4096 bf16", "op": "linear", "rows": 8192, "n": 14336, "k": 4096, "dtype": "bf16",
         "train": False},
        # the GPT-2 shaped MLP's first matrix, forward and backward, a ragged batch
        {"name": "linear 4001x6400x1600 f16 train", "op": "linear", "rows": 4001, "n": 6400, "k": 1600,
         "dtype": "f16", "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "distill", "mx4", "linear"])
    if op == "norm":
        cols = _log(rng, 257, 8192)
        rows = _log(rng, 1, min(32768, 16384 * 4096 // cols))
        train = rng.random() < 0.5
        out = "16" if train else rng.choice(["16", "e4m3"])
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["f16", "bf16", "f32"]), "out": out,
                "block": rng.choice([0, 128]) if out == "e4m3" else 0, "train": train}
    if op == "distill":
        cols = _log(rng, 1001, 128256)
        return {"op": op, "rows": _log(rng, 1, min(8192, 2048 * 128256 // cols)), "cols": cols,
                "k": _log(rng, 1, 100), "dtype": rng.choice(["f16", "bf16", "f32"]),
                "temperature": rng.choice([1.0, 2.0, 4.0]), "scale": rng.choice([1.0, 1024.0])}
    if op == "mx4":
        cols = _log(rng, 33, 14336)
        return {"op": op, "rows": _log(rng, 1, min(16384, 14336 * 4096 // cols)), "cols": cols,
                "dtype": rng.choice(["f16", "bf16", "f32"]), "both": rng.random() < 0.5}
    train = rng.random() < 0.4
    k, n = _log(rng, 129, 14336), _log(rng, 129, 14336)
    most = 8192 * 14336 * 4096 // (3 if train else 1)
    return {"op": op, "rows": _log(rng, 1, max(1, min(8192, most // (n * k)))), "n": n, "k": k,
            "dtype": rng.choice(["f16", "bf16"]), "train": train}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)


def prepare(case, seed):
    g, dt = _gen(seed), TYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        # the residual stream is wider spread than a sublayer's output
        s["x"] = _normal(g, rows, cols, std=0.5, dtype=dt)
        s["residual"] = _normal(g, rows, cols, std=2.0, dtype=dt)
        s["weight"] = _normal(g, cols, std=0.2, mean=1.0, dtype=dt)
        if case["train"]:
            s["dy"] = _normal(g, rows, cols, std=1e-2, dtype=dt)
            s["dh"] = _normal(g, rows, cols, std=1e-2, dtype=dt)
    elif case["op"] == "distill":
        rows, cols, k = case["rows"], case["cols"], case["k"]
        z = torch.empty(rows, cols, dtype=dt, device=DEV)
        for i in range(0, rows, 512):
            z[i:i + 512] = _normal(g, min(512, rows - i), cols, std=1.5)
        # one of each of k equal ranges of the vocabulary, so that a row's ids differ
        width = cols // k
        ids = torch.randint(0, width, (rows, k), generator=g, device=DEV) + torch.arange(k, device=DEV) * width
        z.scatter_add_(1, ids, _normal(g, rows, k, std=2.0, mean=4.0, dtype=dt))
        s["teacher"] = _normal(g, rows, k, std=2.0, mean=8.0).sort(1, descending=True).values.to(dt)
        # some rows have fewer than k teacher logits: their last ids are -1
        have = torch.randint(max(1, k // 2), k + 1, (rows, 1), generator=g, device=DEV)
        have = torch.where(torch.rand(rows, 1, generator=g, device=DEV) < 0.2, have, k)
        s["ids"] = torch.where(torch.arange(k, device=DEV) < have, ids, -1)
        # padding tokens weigh nothing
        s["row_weight"] = (torch.rand(rows, generator=g, device=DEV) >= 0.1).float()
        s["row_weight"][0] = 1.0
        s["logits"] = z
        s["grad_scale"] = 1.0 / rows
    elif case["op"] == "mx4":
        x = _normal(g, case["rows"], case["cols"], std=0.02)
        # a few outlying columns, as weights and activations have
        x *= torch.exp(_normal(g, 1, case["cols"], std=0.5))
        s["x"] = x.to(dt)
    else:
        rows, n, k = case["rows"], case["n"], case["k"]
        s["x"] = _normal(g, rows, k, dtype=dt)
        w = _normal(g, n, k, std=0.02, dtype=dt)
        if case["train"]:
            s["w"] = w
            s["dy"] = _normal(g, rows, n, std=1e-2, dtype=dt)
        else:
            # the weight as the gather and the scales' tiling leave it: packed rows, tiled scales
            codes, scale = _codes(w)
            s["w_data"] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
            s["w_scales"] = _tiled(scale)
        # the word in which a product reports a wait that ran out
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ 4-bit matrices, plain
def _blocks(x):
    """x in fp32, its rows padded with zeros to whole blocks of 32."""
    x = x.float()
    pad = -x.shape[1] % 32
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad)], 1)
    return x.view(x.shape[0], -1, 32)


def _scale_bytes(b):
    """The e8m0 byte of each block: floor(log2 max|x|) - 2, plus 127."""
    top = b.abs().amax(2).view(torch.int32) >> 23
    return (top - 2).clamp_(min=0)


def _scale_values(byte):
    return torch.where(byte > 0, byte << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _e2m1(a):
    """|a| rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to even)."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(a / step).mul_(step).clamp_(max=6.0)


def _quantised(x):
    """The values that x's 4-bit form stands for, in fp32, without the padding."""
    b = _blocks(x)
    scale = _scale_values(_scale_bytes(b))[:, :, None]
    v = b / scale
    q = _e2m1(v.abs()).copysign_(v).mul_(scale)
    return q.view(q.shape[0], -1)[:, :x.shape[1]]


def _codes(x):
    """4-bit codes [rows, padded columns] and scale bytes [rows, blocks] of x."""
    b = _blocks(x)
    byte = _scale_bytes(b)
    v = b / _scale_values(byte)[:, :, None]
    a = _e2m1(v.abs())
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= (v < 0).to(torch.uint8) << 3
    return code.view(x.shape[0], -1), byte.to(torch.uint8)


def _tiled(byte):
    """Scale bytes in tiles of 128 rows by 4 blocks: row r and block b of a tile at (r % 32) * 16 + (r // 32) * 4 + b;
    tiles of a row of tiles follow one another, blocks padded to a multiple of 8."""
    r, c = byte.shape
    full = byte.new_zeros(-(-r // 128) * 128, -(-c // 8) * 8)
    full[:r, :c] = byte
    t = full.view(full.shape[0] // 128, 4, 32, full.shape[1] // 4, 4)
    return t.permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _weights(s):
    """The fp32 values of the packed weight [n, k]."""
    n, k = s["n"], s["k"]
    blocks = -(-k // 32)
    data = s["w_data"].view(n, -1).int()
    code = torch.stack([data & 15, data >> 4], 2).view(n, -1)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=data.device)
    t = s["w_scales"].int().view(-(-n // 128), -(-blocks // 8) * 2, 32, 4, 4).permute(0, 3, 2, 1, 4)
    byte = t.reshape(-(-n // 128) * 128, -1)[:n, :blocks]
    v = table[code].view(n, blocks, 32) * _scale_values(byte)[:, :, None]
    return v.view(n, -1)[:, :k]


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    dt = s["x"].dtype
    h = (s["x"].float() + s["residual"].float()).to(dt)
    hf, w = h.float(), s["weight"].float()
    rstd = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
    y = hf * rstd * w
    out = {"h": h, "rstd": rstd[:, 0]}
    if s["out"] == "e4m3":
        rows, cols = y.shape
        width = s["block"] or cols
        pad = -cols % width
        b = torch.cat([y, y.new_zeros(rows, pad)], 1).view(rows, -1, width)
        scale = b.abs().amax(2, keepdim=True).clamp(min=2.0 ** -100) / 448.0
        out["y"] = (b / scale).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
        out["y_scale"] = scale[:, :, 0]
    else:
        out["y"] = y.to(dt)
    if s["train"]:
        xh, dy = hf * rstd, s["dy"].float()
        gw = dy * w
        dx = rstd * (gw - xh * (gw * xh).mean(1, keepdim=True)) + s["dh"].float()
        out["dx"], out["dw"] = dx.to(dt), (dy * xh).sum(0).to(dt)
    return out


def _plain_distill(s):
    tau, w = s["temperature"], s["row_weight"][:, None]
    z = s["logits"].float() / tau
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    have = s["ids"] >= 0
    t = torch.where(have, s["teacher"].float() / tau, -math.inf)
    pe = torch.exp(t - t.amax(1, keepdim=True))
    psum = pe.sum(1, keepdim=True)
    p = pe / psum
    logp = t - t.amax(1, keepdim=True) - torch.log(psum)
    ids = s["ids"].clamp(min=0)
    terms = torch.where(have, p * (logp - (z.gather(1, ids) - lse)), 0.0)
    loss = w[:, 0] * tau * tau * terms.sum(1)
    grad = e.div_(total).scatter_add_(1, ids, -p)
    grad *= w * (tau * s["grad_scale"] * s["scale"])
    return {"loss": loss, "lse": lse[:, 0], "dlogits": grad.to(s["logits"].dtype)}


def _plain_mx4(s):
    out = {"rows": _quantised(s["x"]).to(s["x"].dtype)}
    if s["both"]:
        out["columns"] = _quantised(s["x"].t()).to(s["x"].dtype)
    return out


def _plain_linear(s):
    dt = s["x"].dtype
    if not s["train"]:
        return {"y": (_quantised(s["x"]) @ _weights(s).t()).to(dt)}
    x, w, dy = s["x"], s["w"], s["dy"]
    return {"y": (_quantised(x) @ _quantised(w).t()).to(dt),
            "dx": (_quantised(dy) @ _quantised(w.t()).t()).to(dt),
            "dw": (_quantised(dy.t()) @ _quantised(x.t()).t()).to(dt)}


# ------------------------------------------------------------------ the framework's calls
def _own_norm(Z, s):
    rows, cols, x = s["rows"], s["cols"], s["x"]
    h = torch.empty_like(x)
    rstd = torch.empty(rows, device=DEV)
    out = {"h": h, "rstd": rstd}
    if s["out"] == "e4m3":
        y = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
        out["y_scale"] = torch.empty(rows, -(-cols // s["block"]) if s["block"] else 1, device=DEV)
    else:
        y = torch.empty_like(x)
    out["y"] = y
    Z.zero_norm_forward(x, s["residual"], s["weight"], rows, cols, EPS, h, y, out.get("y_scale"), s["block"], rstd)
    if s["train"]:
        out["dx"], out["dw"] = torch.empty_like(x), torch.empty_like(s["weight"])
        ws = torch.empty(Z.zero_norm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)
        Z.zero_norm_backward(s["dy"], h, s["weight"], rows, cols, rstd, s["dh"], out["dx"], out["dw"], 0, ws,
                             ws.numel())
    return out


def _own_distill(Z, s):
    rows = s["rows"]
    out = {"loss": torch.empty(rows, device=DEV), "lse": torch.empty(rows, device=DEV),
           "dlogits": torch.empty_like(s["logits"])}
    Z.zero_distill_loss(s["logits"], rows, s["cols"], s["ids"], s["teacher"], s["k"], None, s["temperature"],
                        s["row_weight"], s["grad_scale"] * s["scale"], None, out["loss"], out["lse"], out["dlogits"])
    return out


def _own_mx4(Z, s):
    x, (rows, cols) = s["x"], s["x"].shape
    q = Z.mx4(rows, cols, device=DEV)
    qt = Z.mx4(cols, rows, device=DEV) if s["both"] else None
    Z.zero_mx4_quantize(x, rows, cols, q, qt)
    out = {"rows": torch.empty_like(x)}
    Z.zero_mx4_dequantize(q, out["rows"])
    if s["both"]:
        out["columns"] = torch.empty(cols, rows, dtype=x.dtype, device=DEV)
        Z.zero_mx4_dequantize(qt, out["columns"])
    return out


def _own_linear(Z, s):
    x, rows, n, k = s["x"], s["rows"], s["n"], s["k"]
    y = torch.empty(rows, n, dtype=x.dtype, device=DEV)
    xq = Z.mx4(rows, k, device=DEV)
    if not s["train"]:
        wq = Z.mx4(n, k, s["w_data"], s["w_scales"])
        Z.zero_mx4_quantize(x, rows, k, xq, None)
        Z.zero_mx4_matmul(xq, wq, 1.0, y, s["status"])
        return {"y": y}
    xt, wq, wt = Z.mx4(k, rows, device=DEV), Z.mx4(n, k, device=DEV), Z.mx4(k, n, device=DEV)
    gq, gt = Z.mx4(rows, n, device=DEV), Z.mx4(n, rows, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(s["w"])
    Z.zero_mx4_quantize(x, rows, k, xq, xt)
    Z.zero_mx4_quantize(s["w"], n, k, wq, wt)
    Z.zero_mx4_quantize(s["dy"], rows, n, gq, gt)
    Z.zero_mx4_matmul(xq, wq, 1.0, y, s["status"])
    Z.zero_mx4_matmul(gq, wt, 1.0, dx, s["status"])
    Z.zero_mx4_matmul(gt, xt, 1.0, dw, s["status"])
    return {"y": y, "dx": dx, "dw": dw}


def run(state):
    if own:
        import zero_dp_partitioned_gb300 as Z
        return {"norm": _own_norm, "distill": _own_distill, "mx4": _own_mx4, "linear": _own_linear}[state["op"]](Z, state)
    return {"norm": _plain_norm, "distill": _plain_distill, "mx4": _plain_mx4, "linear": _plain_linear}[state["op"]](state)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        y = 1 if case["out"] == "e4m3" else size
        scales = 4 * rows * (-(-cols // case["block"]) if case["block"] else 1) if case["out"] == "e4m3" else 0
        by = rows * cols * (3 * size + y) + cols * size + 4 * rows + scales
        if case["train"]:
            # dy and dh read, dx written; h is read again as the backward pass's own input
            by += rows * cols * 4 * size + 2 * cols * size + 4 * rows
        return {"bytes": by, "flops": rows * cols * (18 if case["train"] else 7)}
    if case["op"] == "distill":
        rows, cols, k = case["rows"], case["cols"], case["k"]
        return {"bytes": 2 * size * rows * cols + rows * k * (8 + size) + 12 * rows, "flops": 8 * rows * cols}
    if case["op"] == "mx4":
        n = case["rows"] * case["cols"]
        # read once, written as values once for each orientation
        return {"bytes": n * size * (3 if case["both"] else 2), "flops": 4 * n * (2 if case["both"] else 1)}
    t, n, k = case["rows"], case["n"], case["k"]
    if case["train"]:
        return {"bytes": 4 * (t * k + n * k + t * n), "flops": 6 * t * n * k}
    return {"bytes": 2 * t * k + n * k * 17 / 32 + 2 * t * n, "flops": 2 * t * n * k}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(s):
    dt = s["x"].dtype
    h = (s["x"].double() + s["residual"].double()).to(dt)     # h is what is stored; the norm is the norm of it
    hd, w = h.double(), s["weight"].double()
    n = hd.shape[1]
    r = ((hd ** 2).sum(1) / n + EPS) ** -0.5
    y = torch.einsum("ij,i,j->ij", hd, r, w)
    out = {"h": h.double(), "rstd": r, "y": y}
    if s["out"] == "e4m3":
        width = s["block"] or n
        parts = [y[:, c:c + width] for c in range(0, n, width)]
        scale = torch.stack([torch.maximum(c.max(1).values, -c.min(1).values) for c in parts], 1)
        out["y_scale"] = scale = scale.clamp(min=2.0 ** -100) / 448
        out["y"] = torch.cat([c / scale[:, i:i + 1] for i, c in enumerate(parts)], 1)
    if s["train"]:
        dy = s["dy"].double()
        dot = torch.einsum("ij,ij,j->i", dy, hd, w)
        out["dx"] = r[:, None] * dy * w - hd * (r ** 3 * dot / n)[:, None] + s["dh"].double()
        out["dw"] = torch.einsum("ij,ij,i->j", dy, hd, r)
    return out


def _exact_distill(s):
    tau = s["temperature"]
    z = s["logits"].double() / tau
    lse = torch.logsumexp(z, 1)
    ids, have = s["ids"].clamp(min=0), s["ids"] >= 0
    logp = torch.log_softmax((s["teacher"].double() / tau).masked_fill(~have, -math.inf), 1)
    p = logp.exp()
    logq = z.gather(1, ids) - lse[:, None]
    kl = torch.where(have, p * (logp - logq), torch.zeros_like(p)).sum(1)
    w = s["row_weight"].double()
    grad = (z - lse[:, None]).exp_()
    grad.scatter_add_(1, ids, -p)
    grad *= (w * tau * s["grad_scale"] * s["scale"])[:, None]
    return {"loss": w * tau ** 2 * kl, "lse": lse, "dlogits": grad}


def _power(e):
    """2^e in 64 bits, put together from its bits (a power function need not be exact)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_quantised(x):
    """Blocks of 32 along each row, from the definition: the exponent by frexp, the value by the midpoints it is past."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -cols % 32)).unflatten(1, (-1, 32))
    _, e = torch.frexp(b.abs().amax(2, keepdim=True))
    top = b.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, e - 3, torch.full_like(e, -127)).clamp(min=-127)
    scale = _power(e)
    a = b.abs() / scale
    v = torch.zeros_like(a)
    for mid, gap, even in ((0.25, .5, False), (0.75, .5, True), (1.25, .5, False), (1.75, .5, True), (2.5, 1, False),
                           (3.5, 1, True), (5, 2, False)):
        v += gap * ((a >= mid) if even else (a > mid))
    return (torch.sign(b) * v * scale).flatten(1)[:, :cols]


def _exact_weights(s):
    n, k = s["n"], s["k"]
    r, c = torch.arange(n, device=DEV)[:, None], torch.arange(k, device=DEV)[None, :]
    byte = s["w_data"].view(n, -1)[r, c // 2].int()
    code = torch.where(c % 2 == 1, byte >> 4, byte & 15)
    e, m = (code >> 1) & 3, code & 1
    mag = torch.where(e > 0, (1 + 0.5 * m.double()) * (1 << e >> 1).double(), 0.5 * m.double())
    tiles = -(-(-(-k // 32)) // 8) * 2
    blk = c // 32
    at = ((r // 128) * tiles + blk // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + blk % 4
    return torch.where(code > 7, -mag, mag) * _power(s["w_scales"][at].int() - 127)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "distill":
        return _exact_distill(s)
    if case["op"] == "mx4":
        out = {"rows": _exact_quantised(s["x"])}
        if case["both"]:
            out["columns"] = _exact_quantised(s["x"].t())
        return out
    if not case["train"]:
        return {"y": _exact_quantised(s["x"]) @ _exact_weights(s).t()}
    x, w, dy = s["x"], s["w"], s["dy"]
    return {"y": _exact_quantised(x) @ _exact_quantised(w).t(),
            "dx": _exact_quantised(dy) @ _exact_quantised(w.t()).t(),
            "dw": _exact_quantised(dy.t()) @ _exact_quantised(x.t()).t()}

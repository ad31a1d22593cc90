"""Cases of the block operators: layer norm behind a residual's dropout,
dropout from a counter-based generator, and the gated feed-forward block's two
projections with their activation and product, each in the forms a training or
answering program calls them in.

A case names an operator ("op") and its sizes:

  layernorm  h = dropout(x) + r, y = layernorm(h) w + b; p: the probability of
             dropping (0: no dropout), rdtype: the residual stream's type;
             train: the backward pass too (dr, dx behind the dropout, dw, db)
  dropout    y = dropout(x), residual: + r; without one it is also the backward
             pass.  The mask is never stored: element c of row r is kept by the
             16-bit half c % 8 of Philox4x32-10's four words, its key the seed,
             its counter (unit, site, step) with unit = r ceil(cols / 8) + c / 8
  gated      h = act(x Wg^T) (x Wu^T); train: the projections are kept too, and
             dh gives their gradients (stored in 16 bits), dx, dWg and dWu
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token of the GPT-2 shaped model, answering: latency
        {"name": "layernorm 1x1600 f16", "op": "layernorm", "rows": 1, "cols": 1600, "dtype": "f16", "rdtype": "f16",
         "p": 0.0, "train": False},
        # a micro-batch's training pass of the same model, with its dropout
        {"name": "layernorm 8192x1600 bf16 drop train", "op": "layernorm", "rows": 8192, "cols": 1600,
         "dtype": "bf16", "rdtype": "bf16", "p": 0.1, "train": True},
        # the 7.5B GPT-like shape, the residual stream held in fp32, an evaluation's large batch
        {"name": "layernorm 16384x3456 f16 f32", "op": "layernorm", "rows": 16384, "cols": 3456, "dtype": "f16",
         "rdtype": "f32", "p": 0.0, "train": False},
        # a ragged batch of an odd width: no row but the first on a 16-byte boundary
        {"name": "layernorm 2047x1337 f16 drop train", "op": "layernorm", "rows": 2047, "cols": 1337, "dtype": "f16",
         "rdtype": "f16", "p": 0.1, "train": True},
        # a few tokens behind an attention: latency
        {"name": "dropout 5x1600 f16 residual", "op": "dropout", "rows": 5, "cols": 1600, "dtype": "f16", "p": 0.1,
         "residual": True},
        # the embedding's dropout of a large batch, or the gradient of one
        {"name": "dropout 32768x4096 bf16", "op": "dropout", "rows": 32768, "cols": 4096, "dtype": "bf16", "p": 0.1,
         "residual": False},
        # a ragged batch of an odd width in fp32, onto the residual stream
        {"name": "dropout 4095x6401 f32 residual", "op": "dropout", "rows": 4095, "cols": 6401, "dtype": "f32",
         "p": 0.25, "residual": True},
        # one token through the Llama-3-8B shaped block: its weights are read once
        {"name": "gated 1x4096x14336 bf16", "op": "gated", "rows": 1, "cols": 4096, "ff": 14336, "dtype": "bf16",
         "act": "silu", "train": False},
        # the tokens of a hundred requests at once
        {"name": "gated 100x4096x14336 bf16", "op": "gated", "rows": 100, "cols": 4096, "ff": 14336, "dtype": "bf16",
         "act": "silu", "train": False},
        # a prompt's or an evaluation's batch
        {"name": "gated 8192x4096x14336 bf16", "op": "gated", "rows": 8192, "cols": 4096, "ff": 14336,
         "dtype": "bf16", "act": "silu", "train": False},
        # one micro-batch's training pass
        {"name": "gated 8192x4096x14336 bf16 train", "op": "gated", "rows": 8192, "cols": 4096, "ff": 14336,
         "dtype": "bf16", "act": "silu", "train": True},
        # the GPT-2 width with a gated block of 8/3 of it, cut to 8: a ragged batch's training pass
        {"name": "gated 2001x1600x4264 f16 gelu train", "op": "gated", "rows": 2001, "cols": 1600, "ff": 4264,
         "dtype": "f16", "act": "gelu", "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layernorm", "dropout", "gated"])
    if op == "layernorm":
        cols = _log(rng, 257, 8192)
        dtype = rng.choice(["f16", "bf16", "f32"])
        return {"op": op, "rows": _log(rng, 1, min(32768, 16384 * 3456 // cols)), "cols": cols, "dtype": dtype,
                "rdtype": rng.choice([dtype, "f32"]), "p": rng.choice([0.0, 0.1, 0.25]), "train": rng.random() < 0.6}
    if op == "dropout":
        cols = _log(rng, 129, 16384)
        return {"op": op, "rows": _log(rng, 1, min(32768, 32768 * 4096 // cols // 2)), "cols": cols,
                "dtype": rng.choice(["f16", "bf16", "f32"]), "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                "residual": rng.random() < 0.5}
    cols, ff = _log(rng, 129, 8192), _log(rng, 129, 14336)
    if rng.random() < 0.75:
        cols, ff = -(-cols // 8) * 8, -(-ff // 8) * 8
    return {"op": op, "rows": _log(rng, 1, max(1, min(8192, 8192 * 14336 * 4096 // (cols * ff)))), "cols": cols,
            "ff": ff, "dtype": rng.choice(["f16", "bf16"]), "act": rng.choice(["silu", "gelu"]),
            "train": rng.random() < 0.5}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    out = torch.empty(*shape, dtype=dtype, device=DEV)
    for i in range(0, shape[0], 4096):
        part = out[i:i + 4096]
        part.copy_(torch.randn(*part.shape, generator=g, device=DEV).mul_(std).add_(mean))
    return out


def prepare(case, seed):
    g, dt = _gen(seed), TYPES[case["dtype"]]
    s = dict(case)
    rows, cols = case["rows"], case["cols"]
    if case["op"] in ("layernorm", "dropout"):
        # the mask's seed, the place in the model and the step that a training program holds
        s["seed"], s["site"], s["step"] = (seed * 0x9E3779B97F4A7C15 + 0x1234567) % 2 ** 64, 7 + seed % 64, 1 + seed % 1000
    if case["op"] == "layernorm":
        rt = TYPES[case["rdtype"]]
        # the residual stream is wider spread than a sublayer's output, and off centre
        s["x"] = _normal(g, rows, cols, std=0.5, dtype=dt)
        s["residual"] = _normal(g, rows, cols, std=2.0, mean=0.25, dtype=rt)
        s["weight"] = _normal(g, cols, std=0.2, mean=1.0, dtype=dt)
        s["bias"] = _normal(g, cols, std=0.1, dtype=dt)
        if case["train"]:
            s["dy"] = _normal(g, rows, cols, std=1e-2, dtype=dt)
            s["dh"] = _normal(g, rows, cols, std=1e-2, dtype=rt)
    elif case["op"] == "dropout":
        s["x"] = _normal(g, rows, cols, dtype=dt)
        if case["residual"]:
            s["residual"] = _normal(g, rows, cols, std=2.0, dtype=dt)
    else:
        ff = case["ff"]
        s["x"] = _normal(g, rows, cols, dtype=dt)
        s["gate_w"] = _normal(g, ff, cols, std=0.02, dtype=dt)
        s["up_w"] = _normal(g, ff, cols, std=0.02, dtype=dt)
        if case["train"]:
            s["dh"] = _normal(g, rows, ff, std=1e-2, dtype=dt)
        # the word in which a product reports a wait that ran out
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
MASK = 0xFFFFFFFF


def _keep(s):
    """Truth values [rows, cols]: Philox4x32-10, its 64-bit products in int64 (the sign's bits masked away)."""
    rows, cols = s["rows"], s["cols"]
    n = -(-cols // 8)
    unit = torch.arange(rows * n, dtype=torch.int64, device=DEV)
    a, b = unit & MASK, unit >> 32
    c, d = torch.full_like(unit, s["site"]), torch.full_like(unit, s["step"] & MASK)
    k0, k1 = s["seed"] & MASK, s["seed"] >> 32
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32 & MASK) ^ b ^ k0, q & MASK, (p >> 32 & MASK) ^ d ^ k1, p & MASK
        k0, k1 = k0 + 0x9E3779B9 & MASK, k1 + 0xBB67AE85 & MASK
    half = torch.stack([v >> i & 0xFFFF for v in (a, b, c, d) for i in (0, 16)], 1)
    return half.view(rows, n * 8)[:, :cols] >= _limit(s["p"])


def _limit(p):
    """Halves below it are dropped: p in units of 2^-16."""
    return int(math.floor(p * 65536 + 0.5))


def _dropped(x, keep, p):
    return torch.where(keep, x * (65536.0 / (65536 - _limit(p))), 0.0)


def _plain_layernorm(s):
    dt, rt = s["x"].dtype, s["residual"].dtype
    keep = _keep(s) if s["p"] else None
    x = s["x"].float()
    if s["p"]:
        x = _dropped(x, keep, s["p"])
    h = (x + s["residual"].float()).to(rt)
    hf, w = h.float(), s["weight"].float()
    mean = hf.mean(1, keepdim=True)
    dev = hf - mean
    rstd = torch.rsqrt(dev.square().mean(1, keepdim=True) + EPS)
    xh = dev * rstd
    out = {"h": h, "y": (xh * w + s["bias"].float()).to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["train"]:
        dy = s["dy"].float()
        gw = dy * w
        dr = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) + s["dh"].float()
        out["dr"], out["dw"], out["db"] = dr.to(rt), (dy * xh).sum(0).to(dt), dy.sum(0).to(dt)
        if s["p"]:
            out["dx"] = _dropped(dr, keep, s["p"]).to(dt)
    return out


def _plain_dropout(s):
    y = _dropped(s["x"].float(), _keep(s), s["p"])
    if s["residual"] is not False:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


# what GELU's tanh form takes the sigmoid of: 2 sqrt(2 / pi) (x + 0.044715 x^3)
GELU_A, GELU_B = 2 * math.sqrt(2 / math.pi), 0.044715


def _act(g, name):
    """act(g) and its derivative: both activations are g times a sigmoid."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    s = torch.sigmoid(GELU_A * (g + GELU_B * g * g * g))
    return g * s, s + g * s * (1 - s) * (GELU_A * (1 + 3 * GELU_B * g * g))


def _plain_gated(s):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["gate_w"].float(), s["up_w"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, _ = _act(g, s["act"])
    out = {"h": (a * u).to(dt)}
    if s["train"]:
        out["gate"], out["up"] = g.to(dt), u.to(dt)
        g, u, dh = out["gate"].float(), out["up"].float(), s["dh"].float()      # as they are kept
        a, slope = _act(g, s["act"])
        out["dgate"], out["dup"] = (dh * u * slope).to(dt), (dh * a).to(dt)
        dg, du = out["dgate"].float(), out["dup"].float()
        out["dx"] = (dg @ wg + du @ wu).to(dt)
        out["dgate_w"], out["dup_w"] = (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
    return out


# ------------------------------------------------------------------ the framework's calls
def _own_drop(Z, s):
    return Z.drop(s["p"], s["seed"], s["site"], s["step"]) if s["p"] else None


def _own_layernorm(Z, s):
    rows, cols, x, r = s["rows"], s["cols"], s["x"], s["residual"]
    drop = _own_drop(Z, s)
    h, y = torch.empty_like(r), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    out = {"h": h, "y": y, "mean": mean, "rstd": rstd}
    Z.zero_layernorm_forward(x, r, drop, s["weight"], s["bias"], rows, cols, EPS, h, y, mean, rstd)
    if s["train"]:
        out["dr"], out["dw"], out["db"] = torch.empty_like(r), torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        if drop is not None:
            out["dx"] = torch.empty_like(x)
        ws = torch.empty(Z.zero_layernorm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)
        Z.zero_layernorm_backward(s["dy"], h, s["weight"], rows, cols, mean, rstd, s["dh"], drop, out["dr"],
                                  out.get("dx"), out["dw"], out["db"], 0, ws, ws.numel())
    return out


def _own_dropout(Z, s):
    y = torch.empty_like(s["x"])
    r = s["residual"] if s["residual"] is not False else None
    Z.zero_dropout(s["x"], r, s["rows"], s["cols"], _own_drop(Z, s), y)
    return y


def _own_gated(Z, s):
    rows, cols, ff, x, wg, wu = s["rows"], s["cols"], s["ff"], s["x"], s["gate_w"], s["up_w"]
    act = Z.ZERO_SILU if s["act"] == "silu" else Z.ZERO_GELU_TANH
    wide = [torch.empty(rows, ff, dtype=x.dtype, device=DEV) for _ in range(5 if s["train"] else 1)]
    h, gate, up = wide[:3] if s["train"] else (wide[0], None, None)
    out = {"h": h}
    n = Z.zero_gated_forward_workspace_bytes(x, wg, wu, rows, cols, ff)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    Z.zero_gated_forward(x, wg, wu, rows, cols, ff, act, h, gate, up, ws, n, s["status"])
    if s["train"]:
        dg, du = wide[3:]
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
        n = Z.zero_gated_backward_workspace_bytes(x, wg, wu, dg, du, rows, cols, ff)
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
        Z.zero_gated_backward(s["dh"], gate, up, x, wg, wu, rows, cols, ff, act, dg, du, dx, dwg, dwu, 0, ws, n,
                              s["status"])
        out.update(gate=gate, up=up, dgate=dg, dup=du, dx=dx, dgate_w=dwg, dup_w=dwu)
    return out


def run(state):
    if own:
        import zero_dp_partitioned_gb300 as Z
        return {"layernorm": _own_layernorm, "dropout": _own_dropout, "gated": _own_gated}[state["op"]](Z, state)
    return {"layernorm": _plain_layernorm, "dropout": _plain_dropout, "gated": _plain_gated}[state["op"]](state)


def work(case):
    size, rows, cols = 4 if case["dtype"] == "f32" else 2, case["rows"], case["cols"]
    n = rows * cols
    if case["op"] == "layernorm":
        rsize = 4 if case["rdtype"] == "f32" else 2
        by = n * 2 * (size + rsize) + 2 * cols * size + 8 * rows
        if case["train"]:
            # dy, h and dh read (h as the backward pass's own input), dr written, dx too behind a dropout
            by += n * (size + 3 * rsize + (size if case["p"] else 0)) + 3 * cols * size + 8 * rows
        return {"bytes": by, "flops": n * (24 if case["train"] else 9)}
    if case["op"] == "dropout":
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2 * n}
    ff = case["ff"]
    by, fl = 2 * (n + 2 * ff * cols + rows * ff), 4 * rows * ff * cols
    if case["train"]:
        # gate and up written and read again, dh read, dgate and dup written and read again; x and the weights once
        # more; dx and the weights' gradients written
        by += 2 * (2 * rows * ff + 7 * rows * ff + 2 * n + 4 * ff * cols)
        fl *= 3
    return {"bytes": by, "flops": fl}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_keep(s):
    """The generator from its definition, its products put together from 16-bit pieces."""
    rows, cols = s["rows"], s["cols"]
    n = (cols + 7) // 8
    unit = torch.arange(rows, device=DEV)[:, None] * n + torch.arange(n, device=DEV)[None, :]

    def mul(v, m):
        lo, hi = v.remainder(65536), v.div(65536, rounding_mode="floor")
        ml, mh = m % 65536, m // 65536
        low = lo * ml
        mid = hi * ml + lo * mh + low.div(65536, rounding_mode="floor")     # below 2^34
        return (hi * mh + mid.div(65536, rounding_mode="floor"),
                mid.remainder(65536) * 65536 + low.remainder(65536))

    x = [unit.remainder(2 ** 32), unit.div(2 ** 32, rounding_mode="floor"),
         torch.full_like(unit, s["site"]), torch.full_like(unit, s["step"] % 2 ** 32)]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for r in range(10):
        h0, l0 = mul(x[0], 0xD2511F53)
        h1, l1 = mul(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ ((key[0] + r * 0x9E3779B9) % 2 ** 32), l1,
             h0 ^ x[3] ^ ((key[1] + r * 0xBB67AE85) % 2 ** 32), l0]
    keep = torch.empty(rows, n, 8, dtype=torch.bool, device=DEV)
    for e in range(8):
        piece = x[e // 2].div(65536, rounding_mode="floor") if e % 2 else x[e // 2].remainder(65536)
        keep[:, :, e] = piece >= round(s["p"] * 65536)
    return keep.flatten(1)[:, :cols]


def _exact_layernorm(s):
    x = s["x"].double()
    factor = None
    if s["p"]:
        factor = _exact_keep(s).double() * (65536 / (65536 - round(s["p"] * 65536)))
        x = x * factor
    h = (x + s["residual"].double()).to(s["residual"].dtype)     # h is what is stored; the norm is the norm of it
    hd, w, n = h.double(), s["weight"].double(), s["cols"]
    var, mean = torch.var_mean(hd, 1, correction=0, keepdim=True)
    r = (var + EPS) ** -0.5
    xh = (hd - mean) * r
    out = {"h": x + s["residual"].double(), "y": torch.addcmul(s["bias"].double(), xh, w), "mean": mean[:, 0],
           "rstd": r[:, 0]}
    if s["train"]:
        dy = s["dy"].double()
        # the projection onto what the norm leaves free: away from 1 and from xh
        a, b = (dy @ w / n)[:, None], (torch.einsum("ij,ij,j->i", dy, xh, w) / n)[:, None]
        dr = r * (dy * w - a - b * xh) + s["dh"].double()
        out["dr"], out["dw"], out["db"] = dr, torch.einsum("ij,ij->j", dy, xh), dy.sum(0)
        if s["p"]:
            out["dx"] = dr * factor
    return out


def _exact_act(g, name):
    if name == "silu":
        e = torch.exp(-g.abs())
        s = torch.where(g >= 0, 1 / (1 + e), e / (1 + e))
        return g * s, s * (1 + g * (1 - s))
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + GELU_B * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t ** 2) / 2 * math.sqrt(2 / math.pi) * (1 + 3 * GELU_B * g ** 2)


def _exact_gated(s):
    dt = s["x"].dtype
    x, wg, wu = s["x"].double(), s["gate_w"].double(), s["up_w"].double()
    g, u = x @ wg.t(), x @ wu.t()
    out = {"h": _exact_act(g, s["act"])[0] * u}
    if s["train"]:
        out["gate"], out["up"] = g, u
        g, u, dh = g.to(dt).double(), u.to(dt).double(), s["dh"].double()       # the gradients are of what is kept
        a, slope = _exact_act(g, s["act"])
        dg, du = dh * u * slope, dh * a
        out["dgate"], out["dup"] = dg, du
        dg, du = dg.to(dt).double(), du.to(dt).double()                         # and the products of what is stored
        out["dx"] = torch.addmm(dg @ wg, du, wu)
        out["dgate_w"], out["dup_w"] = (x.t() @ dg).t(), (x.t() @ du).t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layernorm":
        return _exact_layernorm(s)
    if case["op"] == "dropout":
        y = s["x"].double() * _exact_keep(s) * (65536 / (65536 - round(s["p"] * 65536)))
        return y + s["residual"].double() if case["residual"] else y
    return _exact_gated(s)

"""zero_layernorm_forward / zero_layernorm_backward against the formulas in 64
bits, at the sizes, alignments and values where they can go wrong.

Tolerances.  u is the unit roundoff of a type (eps / 2), e = 2^-24.  A sum in
fp32, at most 64 terms in a row per thread and then a tree, is off by less than
96 e of its terms' magnitudes: so is the mean of mean|h|, and h - m with it; the
root halves what the squares' sum is off by.  With X = |xh| + (|h| + mean|h|)
rstd, xh is off by less than 128 e X, y by u of itself and 192 e (X |w| + |b|).
dr's fp32 part is taken of its terms' magnitudes, with X in xh's place, at 256 e.
dw and db add `rows` terms in sequences: (rows + 256) e of the magnitudes."""
import pytest
import torch

import block_helpers as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {t: torch.finfo(t).eps / 2 for t in (F16, BF16, F32)}
E = 2.0 ** -24
TINY = {F16: 2.0 ** -25, BF16: 1e-38, F32: 1e-38}
EPS = 1e-5


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def gen(seed=0):
    return torch.Generator(device=DEV).manual_seed(seed)


def rnd(g, *shape, dtype=F32, std=1.0, mean=0.0, off=0, pad=0):
    """A matrix whose rows start `off` elements into rows that are `pad` longer."""
    t = torch.randn(*shape[:-1], shape[-1] + off + pad, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)
    return t[..., off:off + shape[-1]]


def near(got, ref, dtype, extra=0.0, what=""):
    err = (got.double() - ref).abs()
    lim = ref.abs() * (U[dtype] + 4 * E) + TINY[dtype] + extra
    assert bool((err <= lim).all()), (what, float((err - lim).max()))


class Ref:
    """The norm of a stored h in 64 bits, and the magnitudes that tolerances are taken of."""

    def __init__(self, h, w, b, eps=EPS):
        hd = h.double()
        self.w = torch.ones(h.shape[1], dtype=torch.float64, device=DEV) if w is None else w.double()
        self.b = torch.zeros_like(self.w) if b is None else b.double()
        self.mean = hd.mean(1)
        dev = hd - self.mean[:, None]
        self.rstd = (dev.pow(2).mean(1) + eps).pow(-0.5)
        self.xh = dev * self.rstd[:, None]
        self.mag = hd.abs().mean(1)
        self.X = self.xh.abs() + (hd.abs() + self.mag[:, None]) * self.rstd[:, None]
        self.y = self.xh * self.w + self.b

    def check_forward(self, y, mean, rstd):
        near(y, self.y, y.dtype, 192 * E * (self.X * self.w.abs() + self.b.abs()), "y")
        if mean is not None:
            near(mean, self.mean, F32, 96 * E * self.mag, "mean")
        if rstd is not None:
            # the squares about a mean that is off by d are too many by d^2
            near(rstd, self.rstd, F32, self.rstd * (96 * E + (128 * E * self.mag * self.rstd) ** 2), "rstd")

    def gradients(self, dy, dh):
        g, d = dy.double(), 0.0 if dh is None else dh.double()
        gw = g * self.w
        r = self.rstd[:, None]
        dr = r * (gw - gw.mean(1, keepdim=True) - self.xh * (gw * self.xh).mean(1, keepdim=True)) + d
        a = gw.abs()
        size = r * (a + a.mean(1, keepdim=True) + self.X * (a * self.X).mean(1, keepdim=True)) + (d.abs() if dh is not None else 0)
        return dr, size, (g * self.xh).sum(0), (g.abs() * self.X).sum(0), g.sum(0), g.abs().sum(0)

    def check_backward(self, dy, dh, dr, dx, dw, db, k=None, p=0.0):
        rows = dy.shape[0]
        ref, size, rw, sw, rb, sb = self.gradients(dy, dh)
        if dr is not None:
            near(dr, ref, dr.dtype, 256 * E * size, "dr")
        if dx is not None:
            f = 1.0 if k is None else k.double() * B.scale(p)
            near(dx, ref * f, dx.dtype, 256 * E * size * f, "dx")
        if dw is not None:
            near(dw, rw, dw.dtype, (rows + 256) * E * sw, "dw")
        if db is not None:
            near(db, rb, db.dtype, (rows + 256) * E * sb, "db")


def workspace(Z, cols):
    return torch.empty(Z.zero_layernorm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)


SIZES = [(1, 1), (3, 7), (2, 128), (5, 129), (1, 1600), (33, 1337), (7, 4096), (700, 520), (3, 8193), (2, 16384), (3, 16392),
         (2, 20001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("xt,rt", [(F16, F16), (BF16, BF16), (F32, F32), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_forward_and_backward(Z, rows, cols, xt, rt, off, p):
    g = gen(rows * 31 + cols)
    x, r = rnd(g, rows, cols, dtype=xt, off=off), rnd(g, rows, cols, dtype=rt, std=2.0, mean=0.5, off=off)
    w, b = rnd(g, cols, dtype=xt, off=off, mean=1.0), rnd(g, cols, dtype=xt, off=off)
    h, y, dr, dx = (torch.empty(rows, cols, dtype=t, device=DEV) for t in (rt, xt, rt, xt))
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    drop = Z.drop(p, 77, 3, 8) if p else None
    k = B.keep(rows, cols, p, 77, 3, 8) if p else None
    Z.zero_layernorm_forward(x, r, drop, w, b, rows, cols, EPS, h, y, mean, rstd)
    xd = torch.where(k, x.double() * B.scale(p), 0.0) if p else x.double()
    near(h, xd + r.double(), rt, 2 * E * (xd.abs() + r.double().abs()), "h")
    ref = Ref(h, w, b)
    ref.check_forward(y, mean, rstd)
    dy, dh = rnd(g, rows, cols, dtype=xt, off=off), rnd(g, rows, cols, dtype=rt, off=off)
    dw, db = torch.empty(cols, dtype=xt, device=DEV), torch.empty(cols, dtype=xt, device=DEV)
    ws = workspace(Z, cols)
    Z.zero_layernorm_backward(dy, h, w, rows, cols, mean, rstd, dh, drop, dr, dx, dw, db, 0, ws, ws.numel())
    ref.check_backward(dy, dh, dr, dx, dw, db, k, p)


@pytest.mark.parametrize("cols", [200, 203, 16400])
def test_without_what_may_be_missing(Z, cols):
    g = gen(1)
    x, dy = rnd(g, 9, cols, dtype=BF16), rnd(g, 9, cols, dtype=BF16)
    y, dr, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(9, device=DEV), torch.empty(9, device=DEV)
    Z.zero_layernorm_forward(x, None, None, None, None, 9, cols, EPS, None, y, None, None)
    ref = Ref(x, None, None)
    ref.check_forward(y, None, None)
    Z.zero_layernorm_forward(x, None, None, None, None, 9, cols, EPS, None, y, mean, rstd)
    Z.zero_layernorm_backward(dy, x, None, 9, cols, mean, rstd, None, None, dr, None, None, None, 0, None, 0)
    ref.check_backward(dy, None, dr, None, None, None)
    Z.zero_layernorm_backward(dy, x, None, 9, cols, mean, rstd, None, None, None, dx, None, None, 0, None, 0)
    assert torch.equal(dr, dx)
    db, ws = torch.empty(cols, device=DEV), workspace(Z, cols)
    Z.zero_layernorm_backward(dy, x, None, 9, cols, mean, rstd, None, None, dr, None, None, db, 0, ws, ws.numel())
    ref.check_backward(dy, None, dr, None, None, db)
    # dropout of x alone
    d = Z.drop(0.4, 5)
    h = torch.empty_like(x)
    Z.zero_layernorm_forward(x, None, d, None, None, 9, cols, EPS, h, y, mean, rstd)
    k = B.keep(9, cols, 0.4, 5, 0, 0)
    near(h, torch.where(k, x.double() * B.scale(0.4), 0.0), BF16)
    Z.zero_layernorm_backward(dy, h, None, 9, cols, mean, rstd, None, d, None, dx, None, None, 0, None, 0)
    Ref(h, None, None).check_backward(dy, None, None, dx, None, None, k, 0.4)


@pytest.mark.parametrize("wt", [F16, F32])
def test_weights_of_another_type(Z, wt):
    g = gen(11)
    rows, cols = 20, 520
    x, dy = rnd(g, rows, cols, dtype=BF16), rnd(g, rows, cols, dtype=BF16)
    w, b = rnd(g, cols, dtype=wt, mean=1.0), rnd(g, cols, dtype=wt)
    y, dr, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    Z.zero_layernorm_forward(x, None, None, w, b, rows, cols, EPS, None, y, mean, rstd)
    ref = Ref(x, w, b)
    ref.check_forward(y, mean, rstd)
    dw, db, ws = torch.empty_like(w), torch.empty_like(b), workspace(Z, cols)
    Z.zero_layernorm_backward(dy, x, w, rows, cols, mean, rstd, None, None, dr, None, dw, db, 0, ws, ws.numel())
    ref.check_backward(dy, None, dr, None, dw, db)


@pytest.mark.parametrize("cols", [1, 63, 800, 4096, 12288, 17000])
def test_rows_far_off_zero_and_outlying_columns(Z, cols):
    """fp32 rows at 1000 with a spread of 1, and rows with one column of 10^4: the squares are about the mean."""
    g = gen(12)
    x = rnd(g, 6, cols, mean=1000.0)
    x[3:, 0] = 1e4
    x[5] = 3.0                                       # no spread at all
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    Z.zero_layernorm_forward(x, None, None, None, None, 6, cols, EPS, None, y, mean, rstd)
    Ref(x, None, None).check_forward(y, mean, rstd)


@pytest.mark.parametrize("cols,off", [(200, 0), (203, 1), (16400, 0), (16403, 1)])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_written_over_its_inputs(Z, cols, off, p):
    g = gen(2)
    rows = 40
    x, r, dy, dh = (rnd(g, rows, cols, dtype=BF16, off=off) for _ in range(4))
    w = rnd(g, cols, dtype=BF16)
    drop, out = Z.drop(p, 3) if p else None, []
    for over in (False, True):
        rr, dd, gg = (rnd(g, rows, cols, dtype=BF16, off=off).copy_(t) for t in (r, dh, dy))
        h, dr, dx = (rr, dd, gg) if over else (torch.empty_like(r), torch.empty_like(r), torch.empty_like(r))
        y, mean, rstd, dw, db = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(w), torch.empty_like(w)
        ws = workspace(Z, cols)
        Z.zero_layernorm_forward(x, rr, drop, w, None, rows, cols, EPS, h, y, mean, rstd)
        Z.zero_layernorm_backward(gg, h, w, rows, cols, mean, rstd, dd, drop, dr, dx, dw, db, 0, ws, ws.numel())
        out.append([t.clone() for t in (h, y, mean, rstd, dr, dx, dw, db)])
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [256, 1000, 16400])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_spoils_only_itself(Z, cols, bad):
    g = gen(3)
    x = rnd(g, 6, cols, dtype=BF16)
    x[2, cols // 2] = bad
    y = torch.empty_like(x)
    Z.zero_layernorm_forward(x, None, None, None, None, 6, cols, EPS, None, y, None, None)
    good = [0, 1, 3, 4, 5]
    assert torch.isnan(y[2]).any() and torch.isfinite(y[good]).all()


def test_sums_accumulate_in_a_bucket(Z):
    """Micro-batches add into two unaligned stretches of a gradient bucket."""
    g = gen(4)
    bucket = torch.zeros(1000, dtype=BF16, device=DEV)
    dw, db = bucket[3:133], bucket[133:263]
    rw, rb = torch.zeros(130, dtype=torch.float64, device=DEV), torch.zeros(130, dtype=torch.float64, device=DEV)
    ws = workspace(Z, 130)
    for i, rows in enumerate((17, 1, 3000)):
        h, dy = rnd(g, rows, 130, dtype=BF16), rnd(g, rows, 130, dtype=BF16)
        y, dx, mean, rstd = torch.empty_like(h), torch.empty_like(h), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        Z.zero_layernorm_forward(h, None, None, None, None, rows, 130, EPS, None, y, mean, rstd)
        Z.zero_layernorm_backward(dy, h, None, rows, 130, mean, rstd, None, None, dx, None, dw, db, i > 0, ws, ws.numel())
        _, _, w, sw, b, sb = Ref(h, None, None).gradients(dy, None)
        rw, rb = rw + w, rb + b
        near(dw, rw, BF16, (rows + 256) * E * (sw + rw.abs()))
        near(db, rb, BF16, (rows + 256) * E * (sb + rb.abs()))
        rw, rb = dw.double(), db.double()              # each call rounds once
    assert not bucket[:3].any() and not bucket[263:].any()
    before = bucket.clone()
    empty = (dy[:0], h[:0], None, 0, 130, mean, rstd, None, None, dx[:0], None, dw, db)
    Z.zero_layernorm_backward(*empty, 1, ws, ws.numel())
    assert torch.equal(bucket, before)
    Z.zero_layernorm_backward(*empty, 0, ws, ws.numel())
    assert not bucket.any()


def test_gradient_against_differences(Z):
    """Central differences of L = sum(dy y + dh h) along random directions, in
    fp32: with steps of 2^-6 the third-order term and the rounding of L's terms
    (each within 200 e) over the step both stay below 1e-3 of the terms' norm."""
    g = gen(5)
    rows, cols, step = 4, 300, 2.0 ** -6
    x, r, dy, dh = (rnd(g, rows, cols) for _ in range(4))
    w, b = rnd(g, cols) + 1, rnd(g, cols)
    drop = Z.drop(0.2, 8)
    ws = workspace(Z, cols)
    h, y, dr, dx, dw, db = (torch.empty_like(t) for t in (x, x, x, x, w, w))
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)

    def loss(x, r, w, b):
        Z.zero_layernorm_forward(x, r, drop, w, b, rows, cols, EPS, h, y, mean, rstd)
        return float((dy.double() * y.double() + dh.double() * h.double()).sum())

    loss(x, r, w, b)
    Z.zero_layernorm_backward(dy, h, w, rows, cols, mean, rstd, dh, drop, dr, dx, dw, db, 0, ws, ws.numel())
    grads = [t.double().clone() for t in (dx, dr, dw, db)]
    at = [x, r, w, b]
    for i in range(4):
        for _ in range(3):
            v = torch.randn(at[i].shape, generator=g, device=DEV)
            v = v / v.norm()
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + step * v, at[i] - step * v
            slope = (loss(*up) - loss(*down)) / (2 * step)
            want = float((grads[i] * v.double()).sum())
            assert abs(slope - want) < 1e-3 * float(grads[i].norm() + 1), (i, slope, want)


def test_a_captured_pass(Z):
    """Forward and backward captured once, replayed on new inputs, beside an eager pass with its own workspace."""
    g = gen(6)
    rows, cols = 700, 1600
    chain = torch.frombuffer(bytearray(bytes(Z.chain(step=1))), dtype=torch.uint8).to(DEV)
    drop = Z.drop(0.1, 4, 1, chain_dev=chain)
    x, r, dy, dh = (rnd(g, rows, cols, dtype=BF16) for _ in range(4))
    w, b = rnd(g, cols, dtype=BF16, mean=1.0), rnd(g, cols, dtype=BF16)

    def passes(ws, out):
        h, y, mean, rstd, dr, dx, dw, db = out
        Z.zero_layernorm_forward(x, r, drop, w, b, rows, cols, EPS, h, y, mean, rstd)
        Z.zero_layernorm_backward(dy, h, w, rows, cols, mean, rstd, dh, drop, dr, dx, dw, db, 0, ws, ws.numel())

    def buffers():
        e = torch.empty
        return [e(rows, cols, dtype=BF16, device=DEV), e(rows, cols, dtype=BF16, device=DEV), e(rows, device=DEV),
                e(rows, device=DEV), e(rows, cols, dtype=BF16, device=DEV), e(rows, cols, dtype=BF16, device=DEV),
                e(cols, device=DEV), e(cols, device=DEV)]

    ws1, ws2, o1, o2 = workspace(Z, cols), workspace(Z, cols), buffers(), buffers()
    passes(ws1, o1)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        passes(ws1, o1)
    for step in (2, 3):
        for t in (x, r, dy, dh):
            t.copy_(rnd(g, rows, cols, dtype=BF16))
        chain.copy_(torch.frombuffer(bytearray(bytes(Z.chain(step=step))), dtype=torch.uint8))
        passes(ws2, o2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(o1, o2))
        k = B.keep(rows, cols, 0.1, 4, 1, step)
        near(o1[0], torch.where(k, x.double() * B.scale(0.1), 0.0) + r.double(), BF16, 8 * E)


@pytest.mark.parametrize("cols", [264, 265, 20000])
def test_offsets_past_32_bits(Z, cols):
    """Rows 2^30 elements apart: the last one's bytes lie past 2^32."""
    g = gen(13)
    rows, far = 4, 2 ** 30 + 8
    wide = torch.empty(rows * far, dtype=BF16, device=DEV).view(rows, far)
    x, r, h, y, dy, dh, dr = (wide[:, k * 32768:k * 32768 + cols] for k in range(7))
    for t in (x, r, dy, dh):
        t.copy_(rnd(g, rows, cols, dtype=BF16))
    w, b = rnd(g, cols, dtype=BF16, mean=1.0), rnd(g, cols, dtype=BF16)
    mean, rstd, dw, db, ws = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), torch.empty_like(w), torch.empty_like(w), workspace(Z, cols)
    drop, k = Z.drop(0.2, 5), B.keep(rows, cols, 0.2, 5, 0, 0)
    Z.zero_layernorm_forward(x, r, drop, w, b, rows, cols, EPS, h, y, mean, rstd)
    xd = torch.where(k, x.double() * B.scale(0.2), 0.0)
    near(h, xd + r.double(), BF16, 2 * E * (xd.abs() + r.double().abs()))
    ref = Ref(h, w, b)
    ref.check_forward(y, mean, rstd)
    was = dy.clone()
    Z.zero_layernorm_backward(dy, h, w, rows, cols, mean, rstd, dh, drop, dr, dy, dw, db, 0, ws, ws.numel())
    ref.check_backward(was, dh, dr, dy, dw, db, k, 0.2)


def test_a_bad_row_beside_rows_that_share_its_words(Z):
    """Odd widths: a row's first and last 16 bytes hold the neighbouring rows' elements, which may be infinite."""
    g = gen(14)
    rows, cols = 9, 333
    for dtype in (F16, BF16, F32):
        x, dy = rnd(g, rows, cols, dtype=dtype), rnd(g, rows, cols, dtype=dtype)
        x[4], dy[4] = float("inf"), float("nan")
        y, dr, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        Z.zero_layernorm_forward(x, None, None, None, None, rows, cols, EPS, None, y, mean, rstd)
        Z.zero_layernorm_backward(dy, x, None, rows, cols, mean, rstd, None, None, dr, None, None, None, 0, None, 0)
        keep = [r for r in range(rows) if r != 4]
        assert torch.isfinite(y[keep]).all() and torch.isfinite(dr[keep]).all()
        Ref(x[keep], None, None).check_forward(y[keep], mean[keep], rstd[keep])
        Ref(x[keep], None, None).check_backward(dy[keep], None, dr[keep], None, None, None)

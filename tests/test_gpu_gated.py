"""zero_gated_forward / zero_gated_backward against the formulas in 64 bits.

Tolerances.  u is the unit roundoff of the type (eps / 2).  The products of two
16-bit values are exact in fp32; a sum over k is held in fp32, each of its k /
16 steps rounded or cut within 2^-23 of the running magnitude and a step's own
16 terms within 2^-22 of theirs: it is within (k / 16 + 8) 2^-22 of the sum of
magnitudes (T below).  The sigmoid's exponential and quotient are the fast ones:
s within 2^-20 of itself for arguments below 16, where exp's argument is rounded
to 2^-20, and within |t| 2^-23 more beyond.
  h = v U, v = act(G), |act'| <= 1.2:  u |h| + 1.2 T_G |U| + |v| T_U + 2^-18 |h|
  dup = dh v:  u |dup| + 2^-18 |dup|;  dgate = dh U (s + v (1 - s) d), d <= 1.6 (1 + 0.14 g^2) for
  GELU and 1 for SiLU:  u |dgate| + 2^-18 |dh U| (1 + |v d|) (1 - s is off by as much as s)
  the products of dgate and dup as stored:  u |value| + T."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {t: torch.finfo(t).eps / 2 for t in (F16, BF16, F32)}
TINY = {F16: 2.0 ** -25, BF16: 1e-36, F32: 1e-36}


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def gen(seed=0):
    return torch.Generator(device=DEV).manual_seed(seed)


def rnd(g, *shape, dtype=BF16, std=1.0, off=0, pad=0):
    """A matrix whose rows start `off` elements into rows that are `pad` longer."""
    t = torch.randn(*shape[:-1], shape[-1] + off + pad, generator=g, device=DEV).mul_(std).to(dtype)
    return t[..., off:off + shape[-1]]


def near(got, ref, tol, what):
    err = (got.double() - ref).abs()
    lim = ref.abs() * U[got.dtype] + TINY[got.dtype] + tol
    assert bool((err <= lim).all()), (what, float((err - lim).max()), got.shape)


def total(a, b):
    """a b^T, and what its fp32 sum may be off by."""
    a, b = a.double(), b.double()
    return a @ b.t(), (a.abs() @ b.abs().t()) * ((a.shape[1] / 16 + 8) * 2.0 ** -22)


def act_of(g, act):
    """act(g), its slope, and d."""
    if act == 0:
        s, d = torch.sigmoid(g), torch.ones_like(g)
    else:
        a, b = 2 * math.sqrt(2 / math.pi), 0.044715
        s, d = torch.sigmoid(a * (g + b * g ** 3)), a * (1 + 3 * b * g * g)
    return g * s, s + g * s * (1 - s) * d, d


class Block:
    def __init__(self, Z, x, wg, wu, act):
        self.Z, self.x, self.wg, self.wu, self.act = Z, x, wg, wu, act
        (self.rows, self.cols), self.ff = x.shape, wg.shape[0]
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.dtype = x.dtype

    def new(self, rows, cols):
        return torch.full((rows, cols), 7.0, dtype=self.dtype, device=DEV)

    def ws(self, n):
        return (torch.empty(n, dtype=torch.uint8, device=DEV) if n else None), n

    def forward(self, h=None, gate=None, up=None):
        Z, s = self.Z, (self.rows, self.cols, self.ff)
        h = self.new(self.rows, self.ff) if h is None else h
        n = Z.zero_gated_forward_workspace_bytes(self.x, self.wg, self.wu, *s)
        Z.zero_gated_forward(self.x, self.wg, self.wu, *s, self.act, h, gate, up, *self.ws(n), self.status)
        assert int(self.status) == 0
        return h

    def check_forward(self, h, gate=None, up=None):
        g, tg = total(self.x, self.wg)
        u, tu = total(self.x, self.wu)
        v = act_of(g, self.act)[0]
        near(h, v * u, 1.2 * tg * u.abs() + v.abs() * tu + 1.2 * tg * tu + (v * u).abs() * 2.0 ** -18, "h")
        if gate is not None:
            near(gate, g, tg, "gate")
            near(up, u, tu, "up")

    def backward(self, dh, gate, up, dgate, dup, dx, dwg, dwu, accumulate=0):
        Z, s = self.Z, (self.rows, self.cols, self.ff)
        x, wg, wu = (self.x if dwg is not None else None), *((self.wg, self.wu) if dx is not None else (None, None))
        n = Z.zero_gated_backward_workspace_bytes(x, wg, wu, dgate, dup, *s)
        Z.zero_gated_backward(dh, gate, up, x, wg, wu, *s, self.act, dgate, dup, dx, dwg, dwu, accumulate, *self.ws(n),
                              self.status)
        assert int(self.status) == 0

    def check_slopes(self, dh, gate, up, dgate, dup):
        dh, g, u = dh.double(), gate.double(), up.double()
        v, slope, d = act_of(g, self.act)
        near(dup, dh * v, (dh * v).abs() * 2.0 ** -18, "dup")
        near(dgate, dh * u * slope, (dh * u).abs() * (1 + (v * d).abs()) * 2.0 ** -18, "dgate")

    def check_products(self, dgate, dup, dx, dwg, dwu, old=(0.0, 0.0)):
        if dx is not None:
            a, ta = total(dgate, self.wg.t())
            b, tb = total(dup, self.wu.t())
            # one sum of both halves
            k = (2 * self.ff / 16 + 8) / (self.ff / 16 + 8)
            near(dx, a + b, (ta + tb) * k, "dx")
        for dw, d, o in ((dwg, dgate, old[0]), (dwu, dup, old[1])):
            if dw is not None:
                a, ta = total(d.t(), self.x.t())
                near(dw, a + o, ta + 2.0 ** -23 * (a + o).abs(), "dw")


SIZES = [(1, 8, 8), (2, 1000, 77), (4, 4100, 300), (3, 12288, 131), (4, 12296, 40), (5, 4096, 2051), (2, 24576, 9), (3, 40, 24), (1, 1600, 640), (1, 256, 9000), (9, 130, 9728), (121, 264, 520), (129, 72, 10000), (100, 72, 10000), (128, 200, 20000), (5, 1000, 9800), (2, 129, 65), (17, 64, 128), (100, 136, 304), (257, 200, 129), (300, 1337, 257),
         (513, 520, 1000), (255, 72, 2047)]


@pytest.mark.parametrize("rows,cols,ff", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("off", [0, 1])
def test_forward_and_backward(Z, rows, cols, ff, dtype, act, off):
    g = gen(rows + cols * 7 + ff)
    b = Block(Z, rnd(g, rows, cols, dtype=dtype, off=off), rnd(g, ff, cols, dtype=dtype, std=cols ** -0.5, off=off),
              rnd(g, ff, cols, dtype=dtype, std=cols ** -0.5, off=off), act)
    h, gate, up = b.forward(), b.new(rows, ff), b.new(rows, ff)
    b.check_forward(h)
    assert torch.equal(h, b.forward(rnd(g, rows, ff, dtype=dtype, off=off, pad=3), gate, up))
    b.check_forward(h, gate, up)
    dh = rnd(g, rows, ff, dtype=dtype, off=off)
    dg, du = rnd(g, rows, ff, dtype=dtype, off=off), rnd(g, rows, ff, dtype=dtype, off=off)
    dx, dwg, dwu = b.new(rows, cols), rnd(g, ff, cols, dtype=dtype, off=off), b.new(ff, cols)
    b.backward(dh, gate, up, dg, du, dx, dwg, dwu)
    b.check_slopes(dh, gate, up, dg, du)
    b.check_products(dg, du, dx, dwg, dwu)


@pytest.mark.parametrize("rows,cols,ff", [(2100, 192, 2504), (5000, 64, 1032), (300, 2600, 5000)])
def test_pairs_that_walk_many_tiles(Z, rows, cols, ff):
    g = gen(rows)
    b = Block(Z, rnd(g, rows, cols), rnd(g, ff, cols, std=cols ** -0.5), rnd(g, ff, cols, std=cols ** -0.5), 0)
    gate, up = b.new(rows, ff), b.new(rows, ff)
    h = b.forward(None, gate, up)
    b.check_forward(h, gate, up)
    dh, dg, du = rnd(g, rows, ff), b.new(rows, ff), b.new(rows, ff)
    dx, dwg, dwu = b.new(rows, cols), b.new(ff, cols), b.new(ff, cols)
    b.backward(dh, gate, up, dg, du, dx, dwg, dwu)
    b.check_slopes(dh, gate, up, dg, du)
    b.check_products(dg, du, dx, dwg, dwu)
    again = [b.new(rows, cols), b.new(ff, cols), b.new(ff, cols)]
    b.backward(dh, gate, up, dg, du, *again)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dwg, dwu)))


@pytest.mark.parametrize("off", [0, 1])
def test_gradients_over_what_they_come_from(Z, off):
    """dgate and dup in the places of gate, up and dh; the weights' gradients added to a bucket."""
    g = gen(3)
    rows, cols, ff = 130, 264, 333
    b = Block(Z, rnd(g, rows, cols, off=off), rnd(g, ff, cols, std=0.06), rnd(g, ff, cols, std=0.06), 0)
    gate, up = rnd(g, rows, ff, off=off), rnd(g, rows, ff, off=off)
    b.forward(None, gate, up)
    dh = rnd(g, rows, ff, off=off)
    dg, du, dx = b.new(rows, ff), b.new(rows, ff), b.new(rows, cols)
    for wt in (BF16, F32):
        bucket = rnd(g, 2 * ff * cols + 5, dtype=wt)
        old = bucket.clone()
        dwg, dwu = bucket[5:5 + ff * cols].view(ff, cols), bucket[5 + ff * cols:].view(ff, cols)
        was = dwg.double(), dwu.double()
        b.backward(dh, gate, up, dg, du, dx, dwg, dwu, 1)
        b.check_slopes(dh, gate, up, dg, du)
        b.check_products(dg, du, dx, dwg, dwu, was)
        assert torch.equal(bucket[:5], old[:5])
    for places in ((0, 1), (1, 0), (2, 1)):
        t = [rnd(g, rows, ff, off=off).copy_(s) for s in (gate, up, dh)]
        dx2 = b.new(rows, cols)
        b.backward(t[2], t[0], t[1], t[places[0]], t[places[1]], dx2, None, None)
        assert torch.equal(t[places[0]], dg) and torch.equal(t[places[1]], du) and torch.equal(dx2, dx)


def test_parts_that_are_not_wanted(Z):
    g = gen(4)
    rows, cols, ff = 70, 128, 200
    b = Block(Z, rnd(g, rows, cols), rnd(g, ff, cols, std=0.1), rnd(g, ff, cols, std=0.1), 1)
    gate, up, dh = rnd(g, rows, ff), rnd(g, rows, ff), rnd(g, rows, ff)
    dg, du, dx, dwg, dwu = b.new(rows, ff), b.new(rows, ff), b.new(rows, cols), b.new(ff, cols), b.new(ff, cols)
    b.backward(dh, gate, up, dg, du, None, None, None)
    b.check_slopes(dh, gate, up, dg, du)
    b.backward(dh, gate, up, dg, du, dx, None, None)
    b.check_products(dg, du, dx, None, None)
    b.backward(dh, gate, up, dg, du, None, dwg, dwu)
    b.check_products(dg, du, None, dwg, dwu)


def test_empty_sizes(Z):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    e = lambda r, c: torch.full((r, c), 7.0, dtype=BF16, device=DEV)
    h, gate, up = e(5, 9), e(5, 9), e(5, 9)
    Z.zero_gated_forward(e(5, 0), e(9, 0), e(9, 0), 5, 0, 9, 0, h, gate, up, None, 0, st)
    assert not h.any() and not gate.any() and not up.any()
    Z.zero_gated_forward(e(0, 8), e(9, 8), e(9, 8), 0, 8, 9, 0, e(0, 9), None, None, None, 0, st)
    dx, dwg, dwu = e(5, 8), e(9, 8), e(9, 8)
    Z.zero_gated_backward(e(0, 9), e(0, 9), e(0, 9), e(0, 8), e(9, 8), e(9, 8), 0, 8, 9, 0, e(0, 9), e(0, 9), e(0, 8), dwg, dwu, 1,
                          None, 0, st)
    assert bool((dwg == 7).all()) and bool((dwu == 7).all())
    Z.zero_gated_backward(e(0, 9), e(0, 9), e(0, 9), e(0, 8), e(9, 8), e(9, 8), 0, 8, 9, 0, e(0, 9), e(0, 9), e(0, 8), dwg, dwu, 0,
                          None, 0, st)
    assert not dwg.any() and not dwu.any()
    Z.zero_gated_backward(e(5, 0), e(5, 0), e(5, 0), e(5, 8), e(0, 8), e(0, 8), 5, 8, 0, 0, e(5, 0), e(5, 0), dx, e(0, 8), e(0, 8),
                          0, None, 0, st)
    assert not dx.any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_values_stay_in_their_rows_and_columns(Z, bad):
    g = gen(5)
    rows, cols, ff = 300, 100, 290
    b = Block(Z, rnd(g, rows, cols), rnd(g, ff, cols), rnd(g, ff, cols), 0)
    b.x[270, 99] = bad
    b.wu[5, 3] = bad
    h = b.forward()
    spoilt = torch.zeros(rows, ff, dtype=torch.bool, device=DEV)
    spoilt[270] = True
    spoilt[:, 5] = True
    assert torch.isfinite(h[~spoilt]).all()
    assert not torch.isfinite(h[:, 5]).any()
    assert not torch.isfinite(h[270]).all()


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_extreme_gates(Z, act, dtype):
    """Gates far from zero: the activation is 0 or g, its slope 0 or 1, and nothing overflows on the way."""
    big = 60000.0 if dtype == F16 else 1e30
    gate = torch.tensor([[-big, -200.0, -30.0, -1e-3, 0.0, 1e-3, 30.0, 200.0, big]], device=DEV).to(dtype).repeat(3, 1)
    up, dh = torch.full_like(gate, 0.5), torch.full_like(gate, 0.25)
    x = torch.ones(3, 8, dtype=dtype, device=DEV)
    b = Block(Z, x, torch.ones(9, 8, dtype=dtype, device=DEV), torch.ones(9, 8, dtype=dtype, device=DEV), act)
    dg, du = torch.empty_like(gate), torch.empty_like(gate)
    b.backward(dh, gate, up, dg, du, None, None, None)
    assert torch.isfinite(dg).all() and torch.isfinite(du).all()
    assert bool((dg[:, 6:] == 0.125).all()) and bool((dg[:, :2] == 0).all()) and bool((du[:, :2] == 0).all())
    near(du[:, 6:], 0.25 * gate[:, 6:].double(), 0.0, "du")


def test_gradient_against_differences(Z):
    """Central differences of L = sum(dh h) in 64 bits at the 16-bit inputs, along
    random directions, against the fp16 gradients: the formula's slope is exact
    to the third order of a step of 10^-4, and the gradients' entries are within
    2^-10 of dgate's and dup's rounding and their own."""
    g = gen(6)
    rows, cols, ff = 20, 48, 40
    b = Block(Z, rnd(g, rows, cols, dtype=F16), rnd(g, ff, cols, dtype=F16, std=0.2), rnd(g, ff, cols, dtype=F16, std=0.2), 1)
    gate, up, dh = b.new(rows, ff), b.new(rows, ff), rnd(g, rows, ff, dtype=F16)
    b.forward(None, gate, up)
    out = [b.new(rows, cols), b.new(ff, cols), b.new(ff, cols)]
    b.backward(dh, gate, up, b.new(rows, ff), b.new(rows, ff), *out)
    at = [t.double() for t in (b.x, b.wg, b.wu)]

    def loss(x, wg, wu):
        return float((dh.double() * act_of(x @ wg.t(), 1)[0] * (x @ wu.t())).sum())

    for i in range(3):
        for _ in range(3):
            v = torch.randn(at[i].shape, generator=g, device=DEV).double()
            v = v / v.norm()
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
            slope = (loss(*hi) - loss(*lo)) / 2e-4
            assert abs(slope - float((out[i].double() * v).sum())) < 4e-3 * float(out[i].double().norm())


def test_another_stream_a_captured_pass_and_the_same_bits(Z):
    g = gen(7)
    rows, cols, ff = 600, 320, 704
    b = Block(Z, rnd(g, rows, cols), rnd(g, ff, cols, std=0.06), rnd(g, ff, cols, std=0.06), 0)
    dh = rnd(g, rows, ff)

    def passes(o):
        h, gate, up, dg, du, dx, dwg, dwu, ws = o
        Z.zero_gated_forward(b.x, b.wg, b.wu, rows, cols, ff, 0, h, gate, up, None, 0, b.status)
        Z.zero_gated_backward(dh, gate, up, b.x, b.wg, b.wu, rows, cols, ff, 0, dg, du, dx, dwg, dwu, 0, ws, ws.numel(), b.status)

    def buffers():
        n = Z.zero_gated_backward_workspace_bytes(b.x, b.wg, b.wu, dh, dh, rows, cols, ff)
        assert n                                                # the parts of dx's sum
        return [b.new(rows, ff) for _ in range(5)] + [b.new(rows, cols), b.new(ff, cols), b.new(ff, cols),
                                                      torch.zeros(n, dtype=torch.uint8, device=DEV)]

    o1, o2, o3 = buffers(), buffers(), buffers()
    passes(o1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        passes(o2)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(o1[:8], o2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        passes(o3)
    for _ in range(2):
        b.x.copy_(rnd(g, rows, cols))
        passes(o1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(o1[:8], o3))
    assert int(b.status) == 0


def test_a_wait_that_runs_out_is_reported(Z, monkeypatch):
    g = gen(8)
    for rows, ff in ((9, 700), (9, 9800), (300, 700)):
        b = Block(Z, rnd(g, rows, 1000), rnd(g, ff, 1000), rnd(g, ff, 1000), 0)
        monkeypatch.setenv("ZERO_GB300_SPIN_LIMIT", "0")
        h = b.new(rows, ff)
        Z.zero_gated_forward(b.x, b.wg, b.wu, rows, 1000, ff, 0, h, None, None, None, 0, b.status)
        torch.cuda.synchronize()
        assert int(b.status) == 1
        monkeypatch.delenv("ZERO_GB300_SPIN_LIMIT")
        b.status.zero_()
        b.check_forward(b.forward())


def test_many_passes_one_behind_the_other(Z):
    """Passes that nothing waits between: the products of one start beside the
    slopes' last blocks, one block of a pair well before the other, and pairs of
    the next product on SMs that this one leaves idle."""
    g = gen(9)
    rows, cols, ff = 2001, 512, 1352
    b = Block(Z, rnd(g, rows, cols), rnd(g, ff, cols, std=0.04), rnd(g, ff, cols, std=0.04), 0)
    dh, out = rnd(g, rows, ff), []
    ws = b.ws(Z.zero_gated_backward_workspace_bytes(b.x, b.wg, b.wu, dh, dh, rows, cols, ff))
    for i in range(2):
        o = [b.new(rows, ff) for _ in range(5)] + [b.new(rows, cols), b.new(ff, cols), b.new(ff, cols)]
        h, gate, up, dg, du, dx, dwg, dwu = o
        for _ in range(1 if i == 0 else 500):
            Z.zero_gated_forward(b.x, b.wg, b.wu, rows, cols, ff, 0, h, gate, up, None, 0, b.status)
            Z.zero_gated_backward(dh, gate, up, b.x, b.wg, b.wu, rows, cols, ff, 0, dg, du, dx, dwg, dwu, 0, *ws, b.status)
        torch.cuda.synchronize()
        out.append(o)
    assert int(b.status) == 0
    assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("cols", [8, 300, 4104])
def test_an_infinity_in_the_last_column_of_few_rows(Z, rows, cols):
    """It meets its own column of the weights only: gate and up are infinite with the weights' signs, not NaN."""
    g = gen(10)
    b = Block(Z, rnd(g, rows, cols), rnd(g, 70, cols), rnd(g, 70, cols), 0)
    b.x[0, -1] = float("inf")
    gate, up = b.new(rows, 70), b.new(rows, 70)
    b.forward(None, gate, up)
    assert torch.equal(gate[0].double(), b.wg[:, -1].double() * float("inf"))
    assert torch.equal(up[0].double(), b.wu[:, -1].double() * float("inf"))
    assert torch.isfinite(gate[1:]).all()


@pytest.mark.parametrize("rows", [2, 9])
def test_offsets_past_32_bits(Z, rows):
    """Rows 2^29 elements apart: the last one's bytes lie past 2^32."""
    g = gen(11)
    cols, ff, far = 136, 264, 2 ** 29 + 8
    wide = torch.empty(rows * far, dtype=BF16, device=DEV).view(rows, far)
    x, h = wide[:, 64:64 + cols], wide[:, 1024:1024 + ff]
    x.copy_(rnd(g, rows, cols))
    b = Block(Z, x, rnd(g, ff, cols, std=0.1), rnd(g, ff, cols, std=0.1), 0)
    b.forward(h)
    b.check_forward(h)
    gate, up, dg, du, dx = (wide[:, k * 512:k * 512 + n] for k, n in ((4, ff), (5, ff), (6, ff), (7, ff), (8, cols)))
    gate.copy_(rnd(g, rows, ff))
    up.copy_(rnd(g, rows, ff))
    dh, dwg, dwu = rnd(g, rows, ff), b.new(ff, cols), b.new(ff, cols)
    b.backward(dh, gate, up, dg, du, dx, dwg, dwu)
    b.check_slopes(dh, gate, up, dg, du)
    b.check_products(dg, du, dx, dwg, dwu)


def test_two_streams_at_once(Z):
    """Passes of two sizes on two streams, beside one another, each with its own buffers and workspace."""
    g = gen(12)
    blocks = []
    for rows, cols, ff in ((700, 264, 1000), (90, 512, 3000)):
        b = Block(Z, rnd(g, rows, cols), rnd(g, ff, cols, std=0.05), rnd(g, ff, cols, std=0.05), 1)
        dh = rnd(g, rows, ff)
        ws = b.ws(Z.zero_gated_backward_workspace_bytes(b.x, b.wg, b.wu, dh, dh, rows, cols, ff))
        outs = [[b.new(rows, ff) for _ in range(5)] + [b.new(rows, cols), b.new(ff, cols), b.new(ff, cols)] for _ in range(2)]
        blocks.append((b, dh, ws, outs))

    def passes(b, dh, ws, o):
        h, gate, up, dg, du, dx, dwg, dwu = o
        Z.zero_gated_forward(b.x, b.wg, b.wu, b.rows, b.cols, b.ff, 1, h, gate, up, None, 0, b.status)
        Z.zero_gated_backward(dh, gate, up, b.x, b.wg, b.wu, b.rows, b.cols, b.ff, 1, dg, du, dx, dwg, dwu, 0, *ws, b.status)

    for b, dh, ws, outs in blocks:
        passes(b, dh, ws, outs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(100):
        for s, (b, dh, ws, outs) in zip(streams, blocks):
            with torch.cuda.stream(s):
                passes(b, dh, ws, outs[1])
    torch.cuda.synchronize()
    for b, dh, ws, outs in blocks:
        assert int(b.status) == 0
        assert all(torch.equal(p, q) for p, q in zip(*outs))


# Gates far below zero, where the activation is 10^-8 to 10^-39: SiLU's argument t is the gate, GELU's about 1.6 g (1 + 0.045 g^2).
FAR = {0: [-16.0 - 0.75 * i for i in range(108)], 1: [-3.5 - 0.0625 * i for i in range(118)]}


def far_gates(act, dtype):
    return torch.tensor(FAR[act], device=DEV).to(dtype)


def far_reference(g, act):
    """act(g), its slope, and what either may be off by before its rounding, for g < 0.

    exp(t) is off by (2 + 1.2 |t|) ulps of 2^-23 (its documented error), GELU's t
    by five roundings of 2^-24, which exp turns into |t| 2.5 ulps more; quotient,
    products and d: 8 more.  Below 2^-126 fp32 has steps of 2^-149: half a one in
    exp, in the quotient and in each product, all times |g|, |g d| or what it is
    multiplied with."""
    g = g.double()
    if act == 0:
        t, d = g, torch.ones_like(g)
    else:
        a, b = 2 * math.sqrt(2 / math.pi), 0.044715
        t, d = a * (g + b * g ** 3), a * (1 + 3 * b * g * g)
    s = torch.exp(t) / (1 + torch.exp(t))
    rel, grain = (10 + 4 * t.abs()) * 2.0 ** -23, 2.0 ** -149
    size = s * (1 + (g * d).abs())
    return (g * s, (g * s).abs() * rel + (2 + g.abs()) * grain,
            s + g * s * (1 - s) * d, size * rel + (2 + (g * d).abs()) * 2 * grain)


def near_far(got, ref, tol, what):
    """Half a step of the type, of the smallest ones at least."""
    least = {F16: 2.0 ** -25, BF16: 2.0 ** -134}[got.dtype]
    err, lim = (got.double() - ref).abs(), (ref.abs() + tol) * U[got.dtype] + least + tol
    assert bool((err <= lim).all()), (what, int((err > lim).sum()), float((err / lim).max()))


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_slopes_of_gates_far_below_zero(Z, act, dtype):
    """Against relative bounds, down to the type's smallest numbers, rows that start on 16 bytes and not."""
    for off in (0, 1):
        gate = far_gates(act, dtype)
        n = gate.numel() // 8 * 8
        wide = torch.empty(3, n + 8, dtype=dtype, device=DEV)
        g = wide[:, off:off + n]
        g.copy_(gate[:n])
        up, dh = torch.full_like(g, 0.75), torch.full_like(g, 1.5)
        b = Block(Z, torch.ones(3, 8, dtype=dtype, device=DEV), torch.ones(n, 8, dtype=dtype, device=DEV),
                  torch.ones(n, 8, dtype=dtype, device=DEV), act)
        dg, du = torch.empty_like(g), torch.empty_like(g)
        b.backward(dh, g, up, dg, du, None, None, None)
        v, tv, slope, ts = far_reference(g, act)
        near_far(du, 1.5 * v, 1.5 * tv, "dup")
        near_far(dg, 1.125 * slope, 1.125 * ts, "dgate")


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows", [1, 3, 9, 300])
def test_activations_of_gates_far_below_zero(Z, act, dtype, rows):
    """Weights that make every gate one of the list, exactly, and every up 0.75; few rows, a block alone and pairs."""
    gate = far_gates(act, dtype)
    ff = gate.numel()
    x = torch.zeros(rows, 16, dtype=dtype, device=DEV)
    wg, wu = (torch.zeros(ff, 16, dtype=dtype, device=DEV) for _ in range(2))
    x[:, 0], x[:, 9] = 1, 1
    wg[:, 0], wu[:, 9] = gate, 0.75
    b = Block(Z, x, wg, wu, act)
    h, g, u = b.new(rows, ff), b.new(rows, ff), b.new(rows, ff)
    b.forward(h, g, u)
    assert torch.equal(g, gate.expand(rows, ff)) and bool((u == 0.75).all())
    v, tv, _, _ = far_reference(g, act)
    near_far(h, 0.75 * v, 0.75 * tv, "h")

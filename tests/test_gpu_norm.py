"""zero_norm_forward / zero_norm_backward against the formulas in 64 bits, at
the sizes, alignments and values where they can go wrong.

Tolerances.  u is the unit roundoff of a type (2^-8 bf16, 2^-11 fp16, 2^-24
fp32); e = 2^-24.  A sum of squares in fp32, at most 64 terms in a row per
thread and then a tree, is off by less than 80 e, which the root halves; the
remaining products add a few e: y is within u + 64 e of its value (and half a
step of fp16's subnormals).  dx adds terms that may cancel, so its fp32 part
is taken of the terms' magnitudes.  dw adds `rows` fp32 terms in sequences, so
its fp32 part is at most (rows + 32) e of the sum of magnitudes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E = 2.0 ** -24
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def rnd(g, *shape, dtype=F32, std=1.0, off=0, pad=0):
    """A matrix whose rows start `off` elements into rows that are `pad` longer."""
    t = torch.randn(*shape[:-1], shape[-1] + off + pad, generator=g, device=DEV).mul_(std).to(dtype)
    return t[..., off:off + shape[-1]]


def gen(seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def reference(x, r, w, eps):
    h = x if r is None else (x.double() + r.double()).to(r.dtype)
    hd = h.double()
    rstd = (hd.pow(2).mean(1) + eps).pow(-0.5)
    y = hd * rstd[:, None] * (1.0 if w is None else w.double())
    return h, rstd, y


def near(got, ref, u, tiny, extra=0.0):
    err = (got.double() - ref).abs()
    lim = ref.abs() * (u + 64 * E) + tiny + extra
    assert bool((err <= lim).all()), float((err - lim).max())


SIZES = [(1, 1), (3, 7), (2, 128), (5, 129), (1, 1600), (33, 1337), (7, 4096), (3, 8193), (2, 16384), (3, 16392),
         (2, 20001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("xt,rt", [(F16, F16), (BF16, BF16), (F32, F32), (F16, F32), (BF16, F32)])
@pytest.mark.parametrize("off", [0, 1])
def test_forward_and_backward(Z, rows, cols, xt, rt, off):
    g = gen(rows * 31 + cols)
    x, r = rnd(g, rows, cols, dtype=xt, off=off), rnd(g, rows, cols, dtype=rt, std=2.0, off=off)
    w = rnd(g, cols, dtype=xt, off=off) + 1
    h, y, dx = (torch.empty(rows, cols, dtype=t, device=DEV) for t in (rt, xt, rt))
    rstd = torch.empty(rows, device=DEV)
    Z.zero_norm_forward(x, r, w, rows, cols, 1e-5, h, y, None, 0, rstd)
    hr, rr, yr = reference(x, r, w, 1e-5)
    assert torch.equal(h, hr)
    near(rstd, rr, U[F32], 0)
    near(y, yr, U[xt], TINY[xt])
    dy, dh = rnd(g, rows, cols, dtype=xt, off=off), rnd(g, rows, cols, dtype=rt, off=off)
    dw = torch.empty(cols, dtype=xt, device=DEV)
    ws = torch.empty(Z.zero_norm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)
    Z.zero_norm_backward(dy, h, w, rows, cols, rstd, dh, dx, dw, 0, ws, ws.numel())
    xh, gw = hr.double() * rr[:, None], dy.double() * w.double()
    mean, mag = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
    ref = rr[:, None] * (gw - xh * mean) + dh.double()
    size = rr[:, None] * (gw.abs() + xh.abs() * mag) + dh.double().abs()
    near(dx, ref, U[rt], TINY[rt], size * 128 * E)
    terms = dy.double() * xh
    near(dw, terms.sum(0), U[xt], TINY[xt], terms.abs().sum(0) * (rows + 96) * E)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("off", [0, 1])
def test_eight_bit_output(Z, rows, cols, block, off):
    g = gen(cols + block)
    x = rnd(g, rows, cols, dtype=BF16, off=off)
    if rows > 2:
        x[1] = 0                                       # a row of zeros
    w = rnd(g, cols, dtype=BF16) + 1
    n = -(-cols // block) if block else 1
    y = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(rows, n, device=DEV)
    Z.zero_norm_forward(x, None, w, rows, cols, 1e-6, None, y, scale, block, None)
    _, _, yr = reference(x, None, w, 1e-6)
    width = block or cols
    for i in range(n):
        b = yr[:, i * width:(i + 1) * width]
        s = b.abs().amax(1).clamp(min=2.0 ** -100) / 448
        near(scale[:, i], s, U[F32], 0)
        q = y[:, i * width:(i + 1) * width].double() * scale[:, i:i + 1].double()
        # e4m3 has 4 significant bits (u = 2^-4) and steps of 2^-9 at the bottom, both of the scaled value
        lim = b.abs() * (2.0 ** -4 + 128 * E) + s[:, None] * 2.0 ** -10 * (1 + 128 * E)
        assert bool(((q - b).abs() <= lim).all())
    if rows > 2:
        assert not y[1].double().any()


def test_no_residual_no_weight_no_upstream(Z):
    g = gen(1)
    x, dy = rnd(g, 9, 200, dtype=BF16), rnd(g, 9, 200, dtype=BF16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(9, device=DEV)
    Z.zero_norm_forward(x, None, None, 9, 200, 1e-5, None, y, None, 0, rstd)
    _, rr, yr = reference(x, None, None, 1e-5)
    near(y, yr, U[BF16], 0)
    Z.zero_norm_backward(dy, x, None, 9, 200, rstd, None, dx, None, 0, None, 0)
    xh, gd = x.double() * rr[:, None], dy.double()
    near(dx, rr[:, None] * (gd - xh * (gd * xh).mean(1, keepdim=True)), U[BF16], 0,
         rr[:, None] * (gd.abs() + xh.abs() * (gd * xh).abs().mean(1, keepdim=True)) * 128 * E)


@pytest.mark.parametrize("cols", [200, 16400])
def test_written_over_its_inputs(Z, cols):
    g = gen(2)
    x, r = rnd(g, 5, cols, dtype=BF16), rnd(g, 5, cols, dtype=BF16)
    dy, dh = rnd(g, 5, cols, dtype=BF16), rnd(g, 5, cols, dtype=BF16)
    w = rnd(g, cols, dtype=BF16)
    out = []
    for over in (False, True):
        rr, dd = r.clone(), dh.clone()
        h, dx = (rr, dd) if over else (torch.empty_like(r), torch.empty_like(r))
        y, rstd, dw = torch.empty_like(x), torch.empty(5, device=DEV), torch.empty_like(w)
        ws = torch.empty(Z.zero_norm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)
        Z.zero_norm_forward(x, rr, w, 5, cols, 1e-5, h, y, None, 0, rstd)
        Z.zero_norm_backward(dy, h, w, 5, cols, rstd, dd, dx, dw, 0, ws, ws.numel())
        out.append((h, y, rstd, dx, dw))
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cols", [256, 1000, 16400])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_row_spoils_only_itself(Z, cols, bad):
    g = gen(3)
    x = rnd(g, 6, cols, dtype=BF16)
    x[2, cols // 2] = bad
    y8, scale = torch.empty(6, cols, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(6, 1, device=DEV)
    y = torch.empty_like(x)
    Z.zero_norm_forward(x, None, None, 6, cols, 1e-5, None, y, None, 0, None)
    Z.zero_norm_forward(x, None, None, 6, cols, 1e-5, None, y8, scale, 0, None)
    good = [0, 1, 3, 4, 5]
    assert torch.isnan(y[2]).any() and torch.isnan(scale[2]).all()
    assert torch.isfinite(y[good]).all() and torch.isfinite(y8[good].float()).all()


def test_dw_accumulates_in_a_bucket(Z):
    """Micro-batches add into one unaligned stretch of a gradient bucket."""
    g = gen(4)
    bucket = torch.zeros(1000, dtype=BF16, device=DEV)
    dw, ref = bucket[3:3 + 130], torch.zeros(130, dtype=torch.float64, device=DEV)
    ws = torch.empty(Z.zero_norm_workspace_bytes(130), dtype=torch.uint8, device=DEV)
    for i, rows in enumerate((17, 1, 400)):
        h, dy = rnd(g, rows, 130, dtype=BF16), rnd(g, rows, 130, dtype=BF16)
        rstd, dx = torch.rand(rows, generator=g, device=DEV) + 0.5, torch.empty_like(h)
        Z.zero_norm_backward(dy, h, None, rows, 130, rstd, None, dx, dw, i > 0, ws, ws.numel())
        terms = dy.double() * h.double() * rstd.double()[:, None]
        ref = ref + terms.sum(0)
        near(dw, ref, U[BF16], 0, terms.abs().sum(0) * (rows + 96) * E)
        ref = dw.double()                              # each call rounds once
    assert not bucket[:3].any() and not bucket[133:].any()
    Z.zero_norm_backward(dy[:0], h[:0], None, 0, 130, rstd, None, dx[:0], dw, 1, ws, ws.numel())
    assert torch.equal(dw.double(), ref)
    Z.zero_norm_backward(dy[:0], h[:0], None, 0, 130, rstd, None, dx[:0], dw, 0, ws, ws.numel())
    assert not bucket.any()


def test_gradient_against_differences(Z):
    """Central differences of L = sum(dy y + dh h) along random directions, in
    fp32: with steps of 2^-6 the third-order term and the rounding of L's terms
    (each within 80 e) over the step both stay below 1e-3 of the terms' norm."""
    g = gen(5)
    rows, cols, step = 4, 300, 2.0 ** -6
    x, r, dy, dh = (rnd(g, rows, cols) for _ in range(4))
    w = rnd(g, cols) + 1
    ws = torch.empty(Z.zero_norm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)
    h, y, dx, rstd, dw = (torch.empty_like(t) for t in (x, x, x, x[:, 0].contiguous(), w))

    def loss(x, w):
        Z.zero_norm_forward(x, r, w, rows, cols, 1e-5, h, y, None, 0, rstd)
        return float((dy.double() * y.double() + dh.double() * h.double()).sum())

    loss(x, w)
    Z.zero_norm_backward(dy, h, w, rows, cols, rstd, dh, dx, dw, 0, ws, ws.numel())
    for _ in range(4):
        v, u = rnd(g, rows, cols), rnd(g, cols)
        v, u = v / v.norm(), u / u.norm()
        num = (loss(x + step * v, w) - loss(x - step * v, w)) / (2 * step)
        assert abs(num - float((dx.double() * v.double()).sum())) <= 1e-3 * float(dx.norm())
        num = (loss(x, w + step * u) - loss(x, w - step * u)) / (2 * step)
        assert abs(num - float((dw.double() * u.double()).sum())) <= 1e-3 * float(dw.norm())


def test_offsets_past_32_bits(Z):
    rows, cols = 140000, 16384                        # 2.3e9 elements
    x = torch.empty(rows, cols, dtype=BF16, device=DEV)
    x.fill_(0.5)
    x[-1] = rnd(gen(6), cols, dtype=BF16)
    y, rstd, dx = torch.empty_like(x), torch.empty(rows, device=DEV), torch.empty_like(x)
    Z.zero_norm_forward(x, None, None, rows, cols, 0.0, None, y, None, 0, rstd)
    _, rr, yr = reference(x[-2:], None, None, 0.0)
    near(y[-2:], yr, U[BF16], 0)
    Z.zero_norm_backward(x, x, None, rows, cols, rstd, None, dx, None, 0, None, 0)
    xd = x[-2:].double() * rr[:, None]
    ref = rr[:, None] * (x[-2:].double() - xd * (xd * x[-2:].double()).mean(1, keepdim=True))
    near(dx[-2:], ref, U[BF16], 0, rr[:, None] * x[-2:].double().abs() * 256 * E)


def test_another_stream_and_the_same_bits(Z):
    g = gen(7)
    x, dy = rnd(g, 700, 1030, dtype=F16), rnd(g, 700, 1030, dtype=F16)
    s = torch.cuda.Stream()
    ws = torch.empty(Z.zero_norm_workspace_bytes(1030), dtype=torch.uint8, device=DEV)
    outs = []
    for stream in (torch.cuda.current_stream(), s, s):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            h, y, dx = (torch.empty_like(x) for _ in range(3))
            rstd, dw = torch.empty(700, device=DEV), torch.empty(1030, dtype=F16, device=DEV)
            Z.zero_norm_forward(x * 2, x, None, 700, 1030, 1e-5, h, y, None, 0, rstd)
            Z.zero_norm_backward(dy, h, None, 700, 1030, rstd, None, dx, dw, 0, ws, ws.numel())
        stream.synchronize()
        outs.append((h, y, rstd, dx, dw))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


def test_empty_matrices(Z):
    e = torch.empty(0, 64, dtype=BF16, device=DEV)
    Z.zero_norm_forward(e, e, None, 0, 64, 1e-5, e, e, None, 0, None)
    e = torch.empty(5, 0, dtype=BF16, device=DEV)
    Z.zero_norm_forward(e, None, None, 5, 0, 1e-5, None, e, None, 0, None)


@pytest.mark.parametrize("off", [1, 2, 3, 4, 6, 7])
@pytest.mark.parametrize("xt,rt", [(F16, F16), (F32, F32), (BF16, F32)])
def test_rows_that_start_anywhere(Z, off, xt, rt):
    """Every shift of a row against 16 bytes, each matrix at its own, results inside wider rows; the
    values are those of aligned rows, bit for bit, and nothing beside them is written."""
    g = gen(off)
    for rows, cols in ((3, 40), (5, 1000), (2, 2057)):
        def inside(dtype, o):
            wide = torch.full((rows, cols + 11), 3.0, dtype=dtype, device=DEV)
            return wide, wide[:, o:o + cols]
        x, r, dy, dh = (torch.randn(rows, cols, generator=g, device=DEV).to(t) for t in (xt, rt, xt, rt))
        w = torch.randn(cols, generator=g, device=DEV).to(xt)
        res = []
        for o in (None, off):
            ins, outs = [], []
            for t, v, k in ((xt, x, 0), (rt, r, 1), (xt, dy, 2), (rt, dh, 0)):
                wide, m = inside(t, 0 if o is None else (o + k) % 8)
                m.copy_(v)
                ins.append(m if o is not None else v.clone())
            shapes = ((rt, 1), (xt, 0), (rt, 2), (torch.float8_e4m3fn, 3))
            for t, k in shapes:
                if o is None:
                    outs.append((None, torch.empty(rows, cols, dtype=t, device=DEV), 0))
                else:
                    at = (o + k) % 8
                    outs.append((*inside(t, at), at))
            h, y, dx, y8 = (m for _, m, _ in outs)
            rstd, scale = torch.empty(rows, device=DEV), torch.empty(rows, -(-cols // 128), device=DEV)
            Z.zero_norm_forward(ins[0], ins[1], w, rows, cols, 1e-5, h, y, None, 0, rstd)
            Z.zero_norm_forward(ins[0], ins[1], w, rows, cols, 1e-5, None, y8, scale, 128, None)
            Z.zero_norm_backward(ins[2], h, w, rows, cols, rstd, ins[3], dx, None, 0, None, 0)
            for wide, m, at in outs:
                if wide is not None:
                    assert bool((wide[:, :at].float() == 3).all()) and bool((wide[:, at + cols:].float() == 3).all())
            res.append([m.float().clone() for _, m, _ in outs] + [rstd, scale])
        for a, b in zip(*res):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows,cols", [(3, 7), (300, 1337), (2000, 4096), (40, 8200), (3, 20001)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("block", [0, 128])
def test_eight_bit_output_is_the_quotient_rounded(Z, rows, cols, dtype, block):
    """Bit for bit: y in fp32 by the stored rstd, the scale its block's largest magnitude times 1 / 448, and the
    stored value the correctly rounded quotient of the two, rounded to nearest (16-bit weights make many a quotient
    an exact tie).  An infinite weight makes its blocks' scales infinite and their other values 0."""
    g = gen(rows + cols + block)
    x, r, w = rnd(g, rows, cols, dtype=dtype), rnd(g, rows, cols, dtype=dtype, std=2.0), rnd(g, cols, dtype=dtype) + 1
    x[rows // 2], r[rows // 2] = 0, 0
    width = block or cols
    n = -(-cols // width)
    h, rstd = torch.empty_like(x), torch.empty(rows, device=DEV)
    y8, scale = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(rows, n, device=DEV)
    for _ in range(2):
        Z.zero_norm_forward(x, r, w, rows, cols, 1e-5, h, y8, scale, block, rstd)
        y = h.float() * rstd[:, None] * w.float()
        b = torch.nn.functional.pad(y, (0, -cols % width)).view(rows, n, width)
        top = b.abs().amax(2).clamp(min=2.0 ** -100)
        q = (b / scale[:, :, None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
        for got, ref in ((scale, top * torch.full_like(top, 1 / 448)), (y8.float(), q.float())):
            assert torch.equal(torch.isnan(got), torch.isnan(ref))
            assert torch.equal(torch.where(torch.isnan(got), 0.0, got), torch.where(torch.isnan(ref), 0.0, ref))
        w[cols // 2] = float("inf")
        h[rows // 2], x[rows // 2] = 1, 1                 # 0 times infinity is not a number


@pytest.mark.parametrize("rows,cols", [(12000, 1030), (12000, 1032), (5000, 4096), (3000, 8200), (2000, 8199), (1000, 20001)])
@pytest.mark.parametrize("xt,rt", [(F16, F16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("off", [0, 1])
def test_blocks_that_walk_many_rows(Z, rows, cols, xt, rt, off):
    """Several rows a block, none like another: shared memory and the threads' part of dw are used again and again.
    h over the residual, dx over dh, and an e4m3 y beside the 16-bit one."""
    g = gen(rows + cols + off)
    x, r = rnd(g, rows, cols, dtype=xt, off=off), rnd(g, rows, cols, dtype=rt, std=2.0, off=off)
    r *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device=DEV).float()).to(rt)
    w = rnd(g, cols, dtype=xt, off=off) + 1
    hr, rr, yr = reference(x, r, w, 1e-5)
    n = -(-cols // 128)
    y8, scale = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(rows, n, device=DEV)
    y, rstd = torch.empty(rows, cols, dtype=xt, device=DEV), torch.empty(rows, device=DEV)
    Z.zero_norm_forward(x, r, w, rows, cols, 1e-5, None, y8, scale, 128, None)
    Z.zero_norm_forward(x, r, w, rows, cols, 1e-5, r, y, None, 0, rstd)
    assert torch.equal(r, hr)
    near(rstd, rr, U[F32], 0)
    near(y, yr, U[xt], TINY[xt])
    q = hr.float() * rstd[:, None] * w.float()
    b = torch.nn.functional.pad(q, (0, -cols % 128)).view(rows, n, 128)
    assert torch.equal(scale, b.abs().amax(2).clamp(min=2.0 ** -100) * torch.full_like(scale, 1 / 448))
    q = (b / scale[:, :, None]).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    assert torch.equal(y8.view(torch.uint8), q.view(torch.uint8))
    del y, y8, q, b, yr
    dy, dh = rnd(g, rows, cols, dtype=xt, off=off), rnd(g, rows, cols, dtype=rt, off=off)
    xh, gw = hr.double() * rr[:, None], dy.double() * w.double()
    mean, mag = (gw * xh).mean(1, keepdim=True), (gw * xh).abs().mean(1, keepdim=True)
    ref = rr[:, None] * (gw - xh * mean) + dh.double()
    size = rr[:, None] * (gw.abs() + xh.abs() * mag) + dh.double().abs()
    dw = torch.empty(cols, dtype=F32, device=DEV)
    ws = torch.empty(Z.zero_norm_workspace_bytes(cols), dtype=torch.uint8, device=DEV)
    Z.zero_norm_backward(dy, r, w, rows, cols, rstd, dh, dh, dw, 0, ws, ws.numel())
    near(dh, ref, U[rt], TINY[rt], size * 128 * E)
    terms = dy.double() * xh
    near(dw, terms.sum(0), U[F32], TINY[F32], terms.abs().sum(0) * (rows + 96) * E)

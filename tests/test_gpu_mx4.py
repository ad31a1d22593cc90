"""Microscaled 4-bit matrices: quantisation bit for bit, and the product
against 64 bits.

Tolerances.  Quantising is exact.  A product's terms are exact in fp32 (two
values of 2 significant bits and a power of two); the sum over k is held in
fp32, each of its k / 64 steps rounded or cut within 2^-23 of the running
magnitude and a step's own 64 terms within 2^-21 of theirs, so it is within
(k / 64 + 8) 2^-22 of the sum of magnitudes, and D adds its type's rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8, F32: 2.0 ** -24}
VALUES = [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def gen(seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def reference(x):
    """Codes [rows, 32 blocks] and scale bytes [rows, blocks] from the definition."""
    b = torch.nn.functional.pad(x.double(), (0, -x.shape[1] % 32)).unflatten(1, (-1, 32))
    top = b.abs().amax(2)
    bad = ~torch.isfinite(b).all(2)
    top = torch.where(bad, 1.0, top)
    _, e = torch.frexp(top)
    e = torch.where(top > 0, e - 3, -127).clamp(min=-127)
    a = torch.where(bad[:, :, None], 0.0, b.abs()) / power(e)[:, :, None]
    code = torch.zeros_like(a, dtype=torch.int64)
    for mid, up in ((.25, False), (.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5, False)):
        code += (a >= mid) if up else (a > mid)
    code += 8 * torch.signbit(b)
    return code.flatten(1), torch.where(bad, 255, e + 127).to(torch.uint8)


def values(code, byte, cols):
    table = torch.tensor(VALUES, dtype=torch.float64, device=DEV)
    s = power(byte.long() - 127)
    s = torch.where(byte == 255, math.nan, s)
    return (table[code].unflatten(1, (-1, 32)) * s[:, :, None]).flatten(1)[:, :cols]


def unpacked(q, rows, cols):
    """Codes and scale bytes of a quantised matrix as the library wrote it."""
    blocks = -(-cols // 32)
    data, scales = q.tensors
    d = data.view(-1)[:rows * blocks * 16].view(rows, -1).long()
    code = torch.stack([d & 15, d >> 4], 2).flatten(1)
    if q.layout == 0:
        return code, scales.view(-1)[:rows * blocks].view(rows, blocks)
    t = scales.view(-1)[:-(-rows // 128) * -(-cols // 256) * 1024].view(-(-rows // 128), -(-cols // 256) * 2, 32, 4, 4)
    full = t.permute(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)
    assert not full[rows:].any() and not full[:, blocks:].any()          # the padding
    return code, full[:rows, :blocks]


def matrix(g, rows, cols, dtype, off=0):
    x = torch.randn(rows, cols + 2 * off, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-6, 6, x.shape, generator=g, device=DEV).float())
    x = x.to(dtype)[:, off:off + cols]
    if cols >= 40:
        x[0, :32] = 0                                                    # an empty block
        # every tie, and the values that are clipped
        x[-1, :16] = torch.tensor([7.5, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6.5, -.25, -.75, -2.5, -5, -7, 4, -0.0],
                                  device=DEV).to(dtype)
    return x


SIZES = [(1, 1), (1, 32), (3, 33), (31, 31), (32, 64), (65, 1000), (128, 256), (129, 257), (300, 777), (1, 5000),
         (5000, 1), (513, 1600)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("form", ["rows", "columns", "both"])
def test_quantised_bits(Z, rows, cols, dtype, layout, form):
    for off in (0, 1):
        x = matrix(gen(rows + cols), rows, cols, dtype, off)
        q = Z.mx4(rows, cols, layout=layout, device=DEV) if form != "columns" else None
        t = Z.mx4(cols, rows, layout=layout, device=DEV) if form != "rows" else None
        for m in (q, t):
            if m is not None:
                for buf in m.tensors:
                    buf.fill_(0xAA)
        Z.zero_mx4_quantize(x, rows, cols, q, t)
        for m, src in ((q, x), (t, x.t())):
            if m is None:
                continue
            code, byte = unpacked(m, *src.shape)
            rc, rb = reference(src)
            assert torch.equal(byte, rb)
            assert torch.equal(code, rc)
            for dt in (F32, BF16, F16):
                y = torch.empty(src.shape, dtype=dt, device=DEV)
                Z.zero_mx4_dequantize(m, y)
                assert torch.equal(y, values(rc, rb, src.shape[1]).to(dt))


def test_bad_values_stay_visible(Z):
    x = matrix(gen(1), 70, 100, BF16)
    x[3, 40], x[50, 99], x[69, 0] = math.nan, math.inf, -math.inf
    q, t = Z.mx4(70, 100, device=DEV), Z.mx4(100, 70, device=DEV)
    Z.zero_mx4_quantize(x, 70, 100, q, t)
    for m, src in ((q, x), (t, x.t())):
        y = torch.empty(src.shape, dtype=F32, device=DEV)
        Z.zero_mx4_dequantize(m, y)
        bad = ~torch.isfinite(torch.nn.functional.pad(src.float(), (0, -src.shape[1] % 32))).unflatten(1, (-1, 32)).all(2)
        want = bad.repeat_interleave(32, 1)[:, :src.shape[1]]
        assert torch.equal(torch.isnan(y), want) and torch.isfinite(y[~want]).all()


def test_extreme_scales(Z):
    """fp32's smallest and largest: subnormals round at the smallest scale, nothing overflows on the way."""
    x = torch.zeros(4, 64, device=DEV)
    x[0, :4] = torch.tensor([1e-45, 1e-40, 3e-39, 1.2e-38], device=DEV)
    x[1, :4] = torch.tensor([3.4e38, -1e38, 2.1e37, 1.0], device=DEV)
    x[2, 0], x[3, 5] = 1.1754944e-38, 5.9e-39
    q = Z.mx4(4, 64, device=DEV)
    Z.zero_mx4_quantize(x, 4, 64, q, None)
    code, byte = unpacked(q, 4, 64)
    rc, rb = reference(x)
    assert torch.equal(code, rc) and torch.equal(byte, rb)
    y = torch.empty_like(x)
    Z.zero_mx4_dequantize(q, y)
    assert torch.equal(y, values(rc, rb, 64).float())


@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 4100), (128, 256), (300, 96)])
def test_scales_tiled_after_a_gather(Z, rows, cols):
    x = matrix(gen(2), rows, cols, BF16)
    a, b, c = (Z.mx4(rows, cols, layout=l, device=DEV) for l in (0, 1, 1))
    c.tensors[1].fill_(0xFF)
    Z.zero_mx4_quantize(x, rows, cols, a, None)
    Z.zero_mx4_quantize(x, rows, cols, b, None)
    Z.zero_mx4_tile_scales(a, c)
    assert torch.equal(b.tensors[1], c.tensors[1]) and torch.equal(a.tensors[0], b.tensors[0])


def test_a_part_quantised_by_its_owner_and_gathered(Z):
    """Each rank quantises its part of the flat unit; the gathered bytes are those of the whole unit."""
    rows, cols, ranks = 96, 160, 5
    flat = matrix(gen(3), 1, rows * cols, BF16)[0]
    part = rows * cols // ranks
    mine = [Z.mx4(1, part, layout=0, device=DEV) for _ in range(ranks)]
    for r, m in enumerate(mine):
        Z.zero_mx4_quantize(flat[r * part:(r + 1) * part], 1, part, m, None)
    data = torch.empty(rows * cols // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows * cols // 32, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    Z.zero3_gather_bulk([m.tensors[0] for m in mine], [part // 4] * ranks, Z.ZERO_BF16, data, 0, status)
    Z.zero3_gather_segments([m.tensors[1] for m in mine], [part // 64] * ranks, Z.ZERO_BF16, scales)
    whole = Z.mx4(rows, cols, layout=0, device=DEV)
    Z.zero_mx4_quantize(flat.view(rows, cols), rows, cols, whole, None)
    assert torch.equal(data, whole.tensors[0]) and torch.equal(scales, whole.tensors[1])
    assert int(status) == 0


def test_rows_apart(Z):
    """A packed matrix inside a wider one: bytes between the rows are left alone."""
    x = matrix(gen(4), 20, 90, F16)
    buf = torch.full((20, 80), 0x77, dtype=torch.uint8, device=DEV)
    want = Z.mx4(20, 90, device=DEV)
    Z.zero_mx4_quantize(x, 20, 90, want, None)
    scales = torch.empty_like(want.tensors[1])
    q = Z.zero_mx4(buf.data_ptr(), scales.data_ptr(), 20, 90, 80, 1, 0)
    Z.zero_mx4_quantize(x, 20, 90, q, None)
    assert torch.equal(buf[:, :48], want.tensors[0].view(20, 48)) and bool((buf[:, 48:] == 0x77).all())
    d, d2 = torch.empty(20, 20, device=DEV), torch.empty(20, 20, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    Z.zero_mx4_matmul(q, q, 1.0, d, status)
    Z.zero_mx4_matmul(want, want, 1.0, d2, status)
    assert torch.equal(d, d2)


def product(Z, a, b, dtype, alpha=1.0, off=0):
    m, n = a.shape[0], b.shape[0]
    qa, qb = Z.mx4(*a.shape, device=DEV), Z.mx4(*b.shape, device=DEV)
    Z.zero_mx4_quantize(a, *a.shape, qa, None)
    Z.zero_mx4_quantize(b, *b.shape, qb, None)
    d = torch.full((m, n + 2 * off), 7.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    Z.zero_mx4_matmul(qa, qb, alpha, d[:, off:off + n], status)
    assert int(status) == 0
    assert bool((d[:, :off] == 7).all()) and bool((d[:, off + n:] == 7).all())
    va, vb = (values(*reference(x), x.shape[1]) for x in (a, b))
    ref = alpha * (va @ vb.t())
    k = a.shape[1]
    lim = ref.abs() * U[dtype] + abs(alpha) * (va.abs() @ vb.abs().t()) * (k / 64 + 8) * 2.0 ** -22 + \
        (2.0 ** -25 if dtype == F16 else 0)
    err = (d[:, off:off + n].double() - ref).abs()
    assert bool((err <= lim).all()), (float(err.max()), float((err - lim).max()))
    return d


SHAPES = [(1, 1, 1), (1, 128, 32), (1, 300, 4100), (7, 129, 65), (16, 4096, 256), (17, 640, 512), (64, 1000, 1600),
          (65, 257, 300), (128, 128, 128), (129, 128, 33), (200, 90, 700), (256, 256, 1024), (300, 1337, 1337),
          (1000, 520, 96), (2049, 4099, 288)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_product(Z, m, n, k, dtype):
    g = gen(m + n + k)
    a = torch.randn(m, k, generator=g, device=DEV).to(BF16)
    b = torch.randn(n, k, generator=g, device=DEV).to(BF16)
    product(Z, a, b, dtype)
    product(Z, a, b, dtype, alpha=-0.37, off=1)


def test_product_with_scales_that_differ(Z):
    """Scales far apart from block to block and from row to row: every scale meets its own elements."""
    g = gen(9)
    for m, n, k in ((40, 300, 600), (300, 260, 600)):
        a, b = torch.randn(m, k, generator=g, device=DEV), torch.randn(n, k, generator=g, device=DEV)
        a *= torch.exp2(torch.randint(-8, 8, (m, -(-k // 32)), generator=g, device=DEV).float()).repeat_interleave(32, 1)[:, :k]
        b *= torch.exp2(torch.randint(-8, 8, (n, -(-k // 32)), generator=g, device=DEV).float()).repeat_interleave(32, 1)[:, :k]
        product(Z, a, b, F32)


def test_product_keeps_nan(Z):
    g = gen(10)
    for m in (20, 300):
        a, b = torch.randn(m, 500, generator=g, device=DEV), torch.randn(270, 500, generator=g, device=DEV)
        a[3, 499], b[200, 0] = math.inf, math.nan
        qa, qb = Z.mx4(m, 500, device=DEV), Z.mx4(270, 500, device=DEV)
        Z.zero_mx4_quantize(a, m, 500, qa, None)
        Z.zero_mx4_quantize(b, 270, 500, qb, None)
        d, status = torch.empty(m, 270, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
        Z.zero_mx4_matmul(qa, qb, 1.0, d, status)
        want = torch.zeros(m, 270, dtype=torch.bool, device=DEV)
        want[3], want[:, 200] = True, True
        assert torch.equal(torch.isnan(d), want)


def test_linear_layer_gradients(Z):
    """y = x w^T, dx = dy w, dw = dy^T x, each with both operands quantised along its own sum."""
    g = gen(11)
    t, n, k = 333, 480, 290
    x, w, dy = (torch.randn(*s, generator=g, device=DEV).to(BF16) for s in ((t, k), (n, k), (t, n)))
    f = {}
    for name, src in (("x", x), ("w", w), ("dy", dy)):
        f[name], f[name + "t"] = Z.mx4(*src.shape, device=DEV), Z.mx4(*src.shape[::-1], device=DEV)
        Z.zero_mx4_quantize(src, *src.shape, f[name], f[name + "t"])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for p, q, a, b in (("x", "w", x, w), ("dy", "wt", dy, w.t()), ("dyt", "xt", dy.t(), x.t())):
        d = torch.empty(a.shape[0], b.shape[0], device=DEV)
        Z.zero_mx4_matmul(f[p], f[q], 1.0, d, status)
        va, vb = (values(*reference(v), v.shape[1]) for v in (a, b))
        lim = (va.abs() @ vb.abs().t()) * (a.shape[1] / 64 + 8) * 2.0 ** -22
        assert bool(((d.double() - va @ vb.t()).abs() <= lim).all())
    assert int(status) == 0


def test_empty_products(Z):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = torch.full((3, 5), 9.0, device=DEV)
    Z.zero_mx4_matmul(Z.mx4(3, 0, device=DEV), Z.mx4(5, 0, device=DEV), 1.0, d, status)
    assert not d.any()
    Z.zero_mx4_matmul(Z.mx4(0, 64, device=DEV), Z.mx4(5, 64, device=DEV), 1.0, d[:0], status)
    e = torch.empty(0, 7, device=DEV)
    Z.zero_mx4_quantize(e, 0, 7, Z.mx4(0, 7, device=DEV), Z.mx4(7, 0, device=DEV))


def test_offsets_past_32_bits(Z):
    rows, cols = 70000, 32768                                            # 2.3e9 elements
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    x[-3:] = torch.randn(3, cols, generator=gen(12), device=DEV)
    q, t = Z.mx4(rows, cols, device=DEV), Z.mx4(cols, rows, device=DEV)
    Z.zero_mx4_quantize(x, rows, cols, q, t)
    y = torch.empty_like(x)
    Z.zero_mx4_dequantize(q, y)
    assert torch.equal(y[-3:], values(*reference(x[-3:]), cols).to(BF16)) and not y[:-3].any()
    yt = torch.empty(cols, rows, dtype=BF16, device=DEV)
    Z.zero_mx4_dequantize(t, yt)
    assert torch.equal(yt[-5:, -40:], values(*reference(x[-48:, -5:].t()), 48).to(BF16)[:, -40:])
    del y, yt, x, t
    b = torch.randn(32800, 64, generator=gen(13), device=DEV)            # a product of 2.3e9 results
    a = torch.randn(70000, 64, generator=gen(14), device=DEV)
    qa, qb = Z.mx4(70000, 64, device=DEV), Z.mx4(32800, 64, device=DEV)
    Z.zero_mx4_quantize(a, 70000, 64, qa, None)
    Z.zero_mx4_quantize(b, 32800, 64, qb, None)
    d, status = torch.empty(70000, 32800, dtype=BF16, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    Z.zero_mx4_matmul(qa, qb, 1.0, d, status)
    ref = values(*reference(a[-2:]), 64) @ values(*reference(b), 64).t()
    mag = values(*reference(a[-2:]), 64).abs() @ values(*reference(b), 64).abs().t()
    assert bool(((d[-2:].double() - ref).abs() <= ref.abs() * U[BF16] + mag * 9 * 2.0 ** -22).all())


def test_another_stream_and_the_same_bits(Z):
    g = gen(15)
    a, b = torch.randn(700, 900, generator=g, device=DEV), torch.randn(1500, 900, generator=g, device=DEV)
    s = torch.cuda.Stream()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for stream in (torch.cuda.current_stream(), s, s):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            qa, qb = Z.mx4(700, 900, device=DEV), Z.mx4(1500, 900, device=DEV)
            d = torch.empty(700, 1500, device=DEV)
            Z.zero_mx4_quantize(a * 2, 700, 900, qa, None)
            Z.zero_mx4_quantize(b, 1500, 900, qb, None)
            Z.zero_mx4_matmul(qa, qb, 1.0, d, status)
        stream.synchronize()
        outs.append(d)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and int(status) == 0


@pytest.mark.parametrize("m", [8, 300])
def test_a_wait_that_runs_out_is_reported(Z, monkeypatch, m):
    """With a limit of 0 tries every wait gives up at once: the call ends, says so, and the next one is right."""
    g = gen(16)
    a, b = torch.randn(m, 3000, generator=g, device=DEV), torch.randn(700, 3000, generator=g, device=DEV)
    qa, qb = Z.mx4(m, 3000, device=DEV), Z.mx4(700, 3000, device=DEV)
    Z.zero_mx4_quantize(a, m, 3000, qa, None)
    Z.zero_mx4_quantize(b, 700, 3000, qb, None)
    d, status = torch.empty(m, 700, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    monkeypatch.setenv("ZERO_GB300_SPIN_LIMIT", "0")
    Z.zero_mx4_matmul(qa, qb, 1.0, d, status)
    torch.cuda.synchronize()
    assert int(status) == 1
    monkeypatch.delenv("ZERO_GB300_SPIN_LIMIT")
    status.zero_()
    product(Z, a, b, F32)


@pytest.mark.parametrize("m,n,k", [(1, 500, 14000), (5, 2001, 12001), (40, 130, 9001), (100, 300, 8000),
                                   (129, 700, 9000), (300, 600, 14336), (16, 4096, 7168)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_whose_sum_is_shared(Z, m, n, k, dtype):
    """Few tiles and a long sum: clusters of 2, 4 or 8 blocks share it, and add in the order of k."""
    g = gen(m + n + k)
    a, b = torch.randn(m, k, generator=g, device=DEV).to(BF16), torch.randn(n, k, generator=g, device=DEV).to(BF16)
    one = product(Z, a, b, dtype)
    assert torch.equal(one, product(Z, a, b, dtype))
    product(Z, a, b, dtype, off=1)


@pytest.mark.parametrize("off", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_rows_that_start_anywhere(Z, off, dtype):
    """Every shift of a row against 16 bytes, in and out, and nothing written beside it."""
    g = gen(off)
    for rows, cols in ((3, 700), (70, 33), (2, 2049)):
        wide = torch.randn(rows, cols + 9, generator=g, device=DEV).to(dtype)
        x = wide[:, off:off + cols]
        q, t = Z.mx4(rows, cols, device=DEV), Z.mx4(cols, rows, device=DEV)
        Z.zero_mx4_quantize(x, rows, cols, q, t)
        for m, src in ((q, x), (t, x.t())):
            code, byte = unpacked(m, *src.shape)
            rc, rb = reference(src)
            assert torch.equal(code, rc) and torch.equal(byte, rb)
        r = Z.mx4(rows, cols, device=DEV)
        Z.zero_mx4_quantize(x, rows, cols, r, None)
        assert torch.equal(r.buffers[0], q.buffers[0])
        out = torch.full((rows, cols + 9), 5.0, dtype=dtype, device=DEV)
        Z.zero_mx4_dequantize(q, out[:, off:off + cols])
        assert torch.equal(out[:, off:off + cols], values(*reference(x), cols).to(dtype))
        assert bool((out[:, :off] == 5).all()) and bool((out[:, off + cols:] == 5).all())


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("rows,cols", [(2000, 7000), (2001, 7001)])
@pytest.mark.parametrize("off", [0, 1])
def test_blocks_that_walk_many_tiles(Z, dtype, rows, cols, off):
    """Several tiles a block and pieces a warp, both ways, along the rows alone, and back."""
    x = matrix(gen(rows + off), rows, cols, dtype, off)
    q, t, r = Z.mx4(rows, cols, device=DEV), Z.mx4(cols, rows, device=DEV), Z.mx4(rows, cols, device=DEV)
    Z.zero_mx4_quantize(x, rows, cols, q, t)
    Z.zero_mx4_quantize(x, rows, cols, r, None)
    assert torch.equal(r.buffers[0], q.buffers[0])
    for m, src in ((q, x), (t, x.t())):
        code, byte = unpacked(m, *src.shape)
        rc, rb = reference(src)
        assert torch.equal(byte, rb) and torch.equal(code, rc)
        y = torch.empty(src.shape, dtype=dtype, device=DEV)
        Z.zero_mx4_dequantize(m, y)
        assert torch.equal(y, values(rc, rb, src.shape[1]).to(dtype))


def test_scales_tiled_by_threads_that_walk(Z):
    rows, cols = 8100, 14400
    x = torch.randn(rows, cols, generator=gen(20), device=DEV).to(BF16)
    a, b, c = (Z.mx4(rows, cols, layout=l, device=DEV) for l in (0, 1, 1))
    c.tensors[1].fill_(0xFF)
    Z.zero_mx4_quantize(x, rows, cols, a, None)
    Z.zero_mx4_quantize(x, rows, cols, b, None)
    Z.zero_mx4_tile_scales(a, c)
    assert torch.equal(b.tensors[1], c.tensors[1])


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 300), (5000, 4100, 96), (3000, 6000, 2500), (10, 70000, 300),
                                   (40, 70000, 700), (100, 70000, 2100)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_of_many_tiles_a_block(Z, m, n, k, dtype):
    """Four tiles a block and more: each accumulator is used again, overlapping ones too."""
    g = gen(m + n + k)
    a, b = torch.randn(m, k, generator=g, device=DEV).to(BF16), torch.randn(n, k, generator=g, device=DEV).to(BF16)
    product(Z, a, b, dtype)

"""zero_dropout against the mask of the generator's definition and the formula
in 64 bits.

Tolerances.  The scale is an fp32 value, off by 2^-24 of itself at most, and so
are the product x scale and the sum with the residual once each; then one
rounding to the type (u = eps / 2): u + 2 * 2^-24 of the value, or half a step of
fp16's subnormals, and 2 * 2^-24 of the product, also where a residual cancels it
(x scale = 7.5, r = -7.4: the sum of 0.1 may be off by 15 * 2^-24), times 1 + u
for the last rounding."""
import pytest
import torch

import block_helpers as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {t: torch.finfo(t).eps / 2 for t in (F16, BF16, F32)}
E = 2.0 ** -24
TINY = {F16: 2.0 ** -25, BF16: 1e-38, F32: 1e-38}


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def gen(seed=0):
    return torch.Generator(device=DEV).manual_seed(seed)


def rnd(g, *shape, dtype=F32, std=1.0, off=0, pad=0):
    """A matrix whose rows start `off` elements into rows that are `pad` longer."""
    t = torch.randn(*shape[:-1], shape[-1] + off + pad, generator=g, device=DEV).mul_(std).to(dtype)
    return t[..., off:off + shape[-1]]


def near(got, ref, dtype, product=0.0):
    err = (got.double() - ref).abs()
    lim = ref.abs() * (U[dtype] + 2 * E) + TINY[dtype] + product * 2 * E * (1 + U[dtype])
    assert bool((err <= lim).all()), float((err - lim).max())


SIZES = [(1, 1), (3, 7), (5, 8), (2, 128), (33, 255), (1, 1600), (7, 4096), (3, 4100), (300, 1337)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("off,pad", [(0, 0), (0, 8), (1, 0)])
@pytest.mark.parametrize("res", [False, True])
def test_values_and_mask(Z, rows, cols, dtype, off, pad, res):
    g = gen(rows * 31 + cols)
    x = rnd(g, rows, cols, dtype=dtype, off=off, pad=pad)
    r = rnd(g, rows, cols, dtype=dtype, std=2.0, off=off, pad=pad) if res else None
    y = rnd(g, rows, cols, dtype=dtype, off=off, pad=pad)
    args = (0.3, 0xFEDCBA9876543210, 11, 5)
    Z.zero_dropout(x, r, rows, cols, Z.drop(*args), y)
    k = B.keep(rows, cols, *args)
    ref = torch.where(k, x.double() * B.scale(0.3), 0.0)
    near(y, ref + r.double() if res else ref, dtype, ref.abs())
    if not res:
        assert torch.equal((y == 0), ~k | (x == 0))


@pytest.mark.parametrize("cols", [64, 333])
def test_what_the_mask_depends_on(Z, cols):
    x = torch.ones(40, cols, device=DEV)

    def mask(*args, rows=40, of=x):
        y = torch.empty(rows, cols, device=DEV)
        Z.zero_dropout(of[:rows], None, rows, cols, Z.drop(0.5, *args), y)
        return y > 0

    base = mask(1, 2, 3)
    assert torch.equal(base, mask(1, 2, 3))
    for other in ((2, 2, 3), (1 + 2 ** 32, 2, 3), (1, 3, 3), (1, 2, 4)):
        assert not torch.equal(base, mask(*other))
    assert torch.equal(base[:7], mask(1, 2, 3, rows=7))                    # a row's mask does not depend on the rows after it
    wide = torch.ones(40, cols + 5, device=DEV)[:, 3:3 + cols]
    assert torch.equal(base, mask(1, 2, 3, of=wide))                       # nor on the row distance


def test_probabilities_of_zero_and_one(Z):
    g = gen(1)
    for cols in (72, 73):
        x, r = rnd(g, 6, cols, dtype=BF16), rnd(g, 6, cols, dtype=BF16)
        y = torch.empty_like(x)
        for p, want in ((0.0, (x.float() + r.float()).to(BF16)), (2.0 ** -18, (x.float() + r.float()).to(BF16)),
                        (1.0, r), (1 - 2.0 ** -18, r)):
            Z.zero_dropout(x, r, 6, cols, Z.drop(p, 7), y)
            assert torch.equal(y, want)
        Z.zero_dropout(x, None, 6, cols, Z.drop(1.0, 7), y)
        assert not y.any()
        Z.zero_dropout(x, None, 6, cols, Z.drop(65535 / 65536, 7), y)      # one in 65536 kept, scaled by 65536
        near(y, torch.where(B.keep(6, cols, 65535 / 65536, 7, 0, 0), x.double() * 65536, 0.0), BF16)


@pytest.mark.parametrize("cols", [80, 81])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_that_are_dropped_do_no_harm(Z, cols, bad):
    g = gen(2)
    k = B.keep(9, cols, 0.5, 3, 0, 0)
    x = torch.where(k, rnd(g, 9, cols), torch.full((9, cols), bad, device=DEV))
    y = torch.empty_like(x)
    Z.zero_dropout(x, None, 9, cols, Z.drop(0.5, 3), y)
    near(y, torch.where(k, x.double() * 2, 0.0), F32)
    x[k] = bad
    Z.zero_dropout(x, None, 9, cols, Z.drop(0.5, 3), y)
    assert not torch.isfinite(y[k]).any() and not y[~k].any()


@pytest.mark.parametrize("cols,off", [(256, 0), (1000, 1), (777, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_written_over_its_inputs(Z, cols, off, dtype):
    g = gen(3)
    x, r = rnd(g, 500, cols, dtype=dtype, off=off), rnd(g, 500, cols, dtype=dtype, off=off)
    y = torch.empty_like(x)
    d = Z.drop(0.2, 5)
    Z.zero_dropout(x, r, 500, cols, d, y)
    for over in (0, 1):
        x2, r2 = rnd(g, 500, cols, dtype=dtype, off=off).copy_(x), rnd(g, 500, cols, dtype=dtype, off=off).copy_(r)
        to = (x2, r2)[over]
        Z.zero_dropout(x2, r2, 500, cols, d, to)
        assert torch.equal(to, y)


def test_columns_beside_the_matrix_stay(Z):
    for dtype in (F16, F32):
        whole = torch.full((9, 200), 7.0, dtype=dtype, device=DEV)
        Z.zero_dropout(torch.ones(9, 101, dtype=dtype, device=DEV), None, 9, 101, Z.drop(0.5, 1), whole[:, 50:151])
        assert bool((whole[:, :50] == 7).all()) and bool((whole[:, 151:] == 7).all())


def test_the_steps_of_a_chain(Z):
    """The step is read when the kernel runs: a captured call draws anew after each applied step."""
    chain = torch.frombuffer(bytearray(bytes(Z.chain(step=4))), dtype=torch.uint8).to(DEV)
    x, y = torch.ones(50, 160, device=DEV), torch.empty(50, 160, device=DEV)
    d = Z.drop(0.25, 9, site=3, step=99, chain_dev=chain)
    Z.zero_dropout(x, None, 50, 160, d, y)
    assert torch.equal(y > 0, B.keep(50, 160, 0.25, 9, 3, 4))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        Z.zero_dropout(x, None, 50, 160, d, y)
    for step in (5, 6, 7):
        chain.copy_(torch.frombuffer(bytearray(bytes(Z.chain(step=step))), dtype=torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y > 0, B.keep(50, 160, 0.25, 9, 3, step))


def test_another_stream_and_many_tiles(Z):
    g = gen(4)
    rows, cols = 3001, 2056
    x, y = rnd(g, rows, cols, dtype=BF16), torch.empty(rows, cols, dtype=BF16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        Z.zero_dropout(x, None, rows, cols, Z.drop(0.1, 1, 2, 3), y)
    torch.cuda.current_stream().wait_stream(s)
    near(y, torch.where(B.keep(rows, cols, 0.1, 1, 2, 3), x.double() * B.scale(0.1), 0.0), BF16)


@pytest.mark.parametrize("cols", [256, 257])
def test_offsets_past_32_bits(Z, cols):
    """Rows 2^29 elements apart: the last one's bytes lie past 2^32."""
    g = gen(5)
    wide = torch.empty(4 * (2 ** 29 + 8), device=DEV).view(4, 2 ** 29 + 8)
    x, y = wide[:, :cols], wide[:, 4096:4096 + cols]
    x.copy_(rnd(g, 4, cols))
    Z.zero_dropout(x, None, 4, cols, Z.drop(0.3, 2), y)
    near(y, torch.where(B.keep(4, cols, 0.3, 2, 0, 0), x.double() * B.scale(0.3), 0.0), F32)


def test_micro_batches_of_one_step(Z):
    """A chain's step is the same for all micro-batches of a step: sites or seeds of their own draw them masks of their
    own, in a captured step too, and the next step draws others again."""
    chain = torch.frombuffer(bytearray(bytes(Z.chain(step=4))), dtype=torch.uint8).to(DEV)
    x, ys = torch.ones(50, 160, device=DEV), [torch.empty(50, 160, device=DEV) for _ in range(4)]
    drops = [Z.drop(0.25, seed, site=site, chain_dev=chain) for seed, site in ((9, 3), (9, 3 + 8), (10, 3), (9, 3))]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for d, y in zip(drops, ys):
            Z.zero_dropout(x, None, 50, 160, d, y)
    masks = []
    for step in (4, 5):
        chain.copy_(torch.frombuffer(bytearray(bytes(Z.chain(step=step))), dtype=torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        for y, (seed, site) in zip(ys, ((9, 3), (9, 11), (10, 3), (9, 3))):
            assert torch.equal(y > 0, B.keep(50, 160, 0.25, seed, site, step))
        assert torch.equal(ys[0], ys[3])                     # the same seed and site: the same elements
        masks += [y > 0 for y in ys[:3]]
    for i in range(6):
        for j in range(i):
            assert not torch.equal(masks[i], masks[j])


@pytest.mark.parametrize("rows,cols,off", [(5, 1600, 0), (300, 640, 0), (77, 2568, 0), (77, 2568, 1), (77, 2569, 0)])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("p", [0.1, 0.25])
def test_product_and_sum_are_each_rounded_to_fp32(Z, rows, cols, off, dtype, p):
    """The bits of the same steps in fp32, one after the other: with p = 1/4 x 4/3 often falls on half a step of bf16 once it
    is rounded, which a product kept whole into the sum would always pass."""
    g = gen(rows + cols)
    x, r = rnd(g, rows, cols, dtype=dtype, off=off), rnd(g, rows, cols, dtype=dtype, std=2.0, off=off)
    y, k = torch.empty_like(x), B.keep(rows, cols, p, 13, 5, 7)
    product = torch.where(k, x.float() * torch.tensor(B.scale(p), dtype=F32, device=DEV), torch.zeros((), device=DEV))
    d = Z.drop(p, 13, 5, 7)
    Z.zero_dropout(x, r, rows, cols, d, y)
    assert torch.equal(y, (product + r.float()).to(dtype)), int((y != (product + r.float()).to(dtype)).sum())
    Z.zero_dropout(x, None, rows, cols, d, y)
    assert torch.equal(y, product.to(dtype))

"""zero_distill_loss / zero_distill_backward against the formulas in 64 bits.

Tolerances.  ex2.approx is within 2^-22; the exponent z k - m k is rounded
within 2^-24 of its size, at most 2^7 here, before it is raised, which makes
2^-17 in the worst case of a term far below the maximum and 2^-20 of the sum.
So q is within 2^-17 (and the type's rounding u); lse within 2^-20 + 2^-23 of
its size; the loss, a p-weighted mean of differences of logarithms, within
2^-19 of the largest logarithm in it, times T^2 w."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def gen(seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def problem(seed, rows, cols, k, dtype, off=0, ids_dtype=torch.int64):
    g = gen(seed)
    z = (torch.randn(rows, cols + 2 * off, generator=g, device=DEV) * 2).to(dtype)[:, off:off + cols]
    ids = torch.rand(rows, cols, generator=g, device=DEV).topk(k, 1).indices.to(ids_dtype) if cols < 200000 else \
        torch.randint(0, cols, (rows, k), generator=g, device=DEV).to(ids_dtype)
    t = (torch.randn(rows, k, generator=g, device=DEV) * 2 + 3).to(dtype)
    return g, z, ids, t


def reference(z, ids, t, tau, w, scale, t_lse=None):
    zd = z.double() / tau
    lse = torch.logsumexp(zd, 1)
    cols = z.shape[1]
    have = (ids >= 0) & (ids < cols) & (t != -math.inf)
    at = torch.where(have, ids, 0).long()
    td = (t.double() / tau).masked_fill(~have, -math.inf)
    logp = td - (torch.logsumexp(td, 1, keepdim=True) if t_lse is None else t_lse.double()[:, None])
    p = torch.where(have, logp.exp(), torch.zeros_like(logp))
    P = p.sum(1, keepdim=True)
    terms = torch.where(have & (p > 0), p * (logp - (zd.gather(1, at) - lse[:, None])), torch.zeros_like(p))
    wd = torch.ones(z.shape[0], dtype=torch.float64, device=DEV) if w is None else w.double()
    q = (zd - lse[:, None]).exp()
    pv = torch.zeros_like(q).scatter_add_(1, at, p)
    dead = (wd == 0) | ~have.any(1)
    loss = torch.where(dead, 0.0, wd * tau * tau * terms.sum(1))
    dz = torch.where(dead[:, None], 0.0, (P * q - pv) * (wd * tau * scale)[:, None])
    mag = (P * q + pv) * (wd * tau * scale).abs()[:, None]
    top = torch.where(have, logp.abs() + (zd.gather(1, at) - lse[:, None]).abs(), 0.0).amax(1) if t.shape[1] else lse * 0
    return loss, lse, dz, mag, top


def check(z, ids, t, tau, w, scale, loss, lse, dz, t_lse=None, lse_in=None):
    rl, rlse, rdz, mag, top = reference(z, ids, t, tau, w, scale, t_lse)
    wd = 1.0 if w is None else w.double().abs()
    if lse is not None:
        assert bool(((lse.double() - rlse).abs() <= 2.0 ** -20 + rlse.abs() * 2.0 ** -23).all())
    if loss is not None:
        lim = 2.0 ** -19 * tau * tau * wd * (1 + top + rlse.abs())
        assert bool(((loss.double() - rl).abs() <= lim).all()), float(((loss.double() - rl).abs() - lim).max())
    if dz is not None:
        tiny = 2.0 ** -25 if z.dtype == F16 else 1e-37
        lim = rdz.abs() * U[z.dtype] + mag * 2.0 ** -17 + tiny
        err = (dz.double() - rdz).abs()
        assert bool((err <= lim).all()), float((err - lim).max())


SIZES = [(1, 1, 1), (2, 9, 3), (5, 1000, 16), (3, 4097, 100), (7, 50257, 33), (2, 128256, 64), (40, 8191, 8),
         (700, 3000, 5), (3, 262144, 4), (2, 300001, 1024)]


@pytest.mark.parametrize("rows,cols,k", SIZES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_loss_and_gradient(Z, rows, cols, k, dtype, off):
    tau = 2.0 if rows % 2 else 1.0
    ids_dtype = torch.int32 if off == 1 else torch.int64
    g, z, ids, t = problem(rows + cols, rows, cols, k, dtype, off, ids_dtype)
    w = torch.rand(rows, generator=g, device=DEV) + 0.1
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dz = torch.empty(rows, cols, dtype=dtype, device=DEV)
    Z.zero_distill_loss(z, rows, cols, ids, t, k, None, tau, w, 0.25, None, loss, lse, dz)
    check(z, ids, t, tau, w, 0.25, loss, lse, dz)
    dz2 = torch.empty(rows, cols, dtype=dtype, device=DEV)
    Z.zero_distill_backward(z, rows, cols, ids, t, k, None, tau, w, 0.25, None, lse, dz2)
    check(z, ids, t, tau, w, 0.25, None, None, dz2)


@pytest.mark.parametrize("cols,dtype", [(50257, F16), (1001, BF16), (300001, F16), (140001, F32)])
@pytest.mark.parametrize("rows", [2, 400])
def test_gradient_over_the_logits(Z, rows, cols, dtype):
    rows = 2 if cols > 100000 and rows > 2 and dtype == F32 else rows
    _, z, ids, t = problem(7, rows, cols, 12, dtype)
    want, loss, lse = torch.empty_like(z), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    Z.zero_distill_loss(z, rows, cols, ids, t, 12, None, 1.0, None, 1.0, None, loss, lse, want)
    over, l2 = z.clone(), torch.empty(rows, device=DEV)
    Z.zero_distill_loss(over, rows, cols, ids, t, 12, None, 1.0, None, 1.0, None, l2, None, over)
    assert torch.equal(over, want) and torch.equal(l2, loss)
    bwd, over = torch.empty_like(z), z.clone()
    Z.zero_distill_backward(z, rows, cols, ids, t, 12, None, 1.0, None, 1.0, None, lse, bwd)
    Z.zero_distill_backward(over, rows, cols, ids, t, 12, None, 1.0, None, 1.0, None, lse, over)
    assert torch.equal(over, bwd)


def test_teachers_own_log_sum_exp(Z):
    g, z, ids, t = problem(8, 6, 2000, 20, F32)
    t_lse = torch.logsumexp(t.double() / 2, 1).float() + 0.3       # the rest of the teacher's vocabulary
    loss, lse, dz = torch.empty(6, device=DEV), torch.empty(6, device=DEV), torch.empty_like(z)
    Z.zero_distill_loss(z, 6, 2000, ids, t, 20, t_lse, 2.0, None, 1.0, None, loss, lse, dz)
    check(z, ids, t, 2.0, None, 1.0, loss, lse, dz, t_lse)


def test_rows_that_count_for_nothing(Z):
    """Weight 0, no entries, entries of -inf, no entries at all (k = 0): loss and
    gradient 0 whatever the logits hold; the others are as without them."""
    _, z, ids, t = problem(9, 6, 5000, 10, BF16)
    z[0], z[1], z[2] = math.nan, math.inf, -math.inf
    z[0, 5] = 1.0
    w = torch.tensor([0.0, 1, 1, 1, 1, 1], device=DEV)
    ids[1] = -1
    t[2] = -math.inf
    ids[3, 4:], ids[3, 0] = -1, 5000               # a ragged list, and an id past the end
    loss, lse, dz = torch.empty(6, device=DEV), torch.empty(6, device=DEV), torch.empty_like(z)
    Z.zero_distill_loss(z, 6, 5000, ids, t, 10, None, 1.0, w, 1.0, None, loss, lse, dz)
    assert not loss[:3].any() and not dz[:3].any()
    check(z[3:], ids[3:], t[3:], 1.0, w[3:], 1.0, loss[3:], lse[3:], dz[3:])
    Z.zero_distill_loss(z, 6, 5000, ids[:, :0], t[:, :0], 0, None, 1.0, w, 1.0, None, loss, None, dz)
    assert not loss.any() and not dz.any()


def test_masked_columns_and_repeated_ids(Z):
    _, z, ids, t = problem(10, 4, 70001, 12, F32)
    z[:, 1000:40000] = -math.inf                   # whole shares of a row masked
    ids = torch.randint(0, 1000, ids.shape, generator=gen(1), device=DEV)
    ids[:, 6:] = ids[:, :6]                        # every id twice
    loss, lse, dz = torch.empty(4, device=DEV), torch.empty(4, device=DEV), torch.empty_like(z)
    Z.zero_distill_loss(z, 4, 70001, ids, t, 12, None, 1.0, None, 1.0, None, loss, lse, dz)
    check(z, ids, t, 1.0, None, 1.0, loss, lse, dz)
    assert not dz[:, 1000:40000].any()
    ids[1, 0] = 2000                               # the teacher wants a masked column
    Z.zero_distill_loss(z, 4, 70001, ids, t, 12, None, 1.0, None, 1.0, None, loss, lse, dz)
    assert loss[1] == math.inf and torch.isfinite(loss[[0, 2, 3]]).all() and torch.isfinite(dz).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("cols", [300, 128256])
def test_a_bad_logit_reaches_its_rows_gradient(Z, bad, cols):
    """So that the step's overflow check sees it."""
    _, z, ids, t = problem(11, 3, cols, 4, BF16)
    z[1, cols - 1] = bad
    loss, dz = torch.empty(3, device=DEV), torch.empty_like(z)
    Z.zero_distill_loss(z, 3, cols, ids, t, 4, None, 1.0, None, 1.0, None, loss, None, dz)
    assert torch.isnan(dz[1].float()).all() and torch.isnan(loss[1])
    assert torch.isfinite(dz[[0, 2]].float()).all() and torch.isfinite(loss[[0, 2]]).all()


def test_loss_scale_from_the_chain(Z):
    _, z, ids, t = problem(12, 8, 600, 6, F32)
    c = Z.chain(loss_scale=1024.0)
    dev = torch.frombuffer(bytearray(bytes(c)), dtype=torch.uint8).to(DEV)
    dz = torch.empty_like(z)
    Z.zero_distill_loss(z, 8, 600, ids, t, 6, None, 1.0, None, 0.125, dev, None, None, dz)
    check(z, ids, t, 1.0, None, 128.0, None, None, dz)
    # captured once, replayed after the chain has lowered S
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        Z.zero_distill_loss(z, 8, 600, ids, t, 6, None, 1.0, None, 0.125, dev, None, None, dz)
    dev.copy_(torch.frombuffer(bytearray(bytes(Z.chain(loss_scale=256.0))), dtype=torch.uint8))
    graph.replay()
    torch.cuda.synchronize()
    check(z, ids, t, 1.0, None, 32.0, None, None, dz)


def test_gradient_against_differences(Z):
    """Central differences of the loss along random directions: a step of 2^-5
    leaves a third-order term below 2^-10 / 6 and a rounding below 2^-15 / 2^-5."""
    g, z, ids, t = problem(13, 3, 400, 6, F32)
    step, tau = 2.0 ** -5, 2.0
    dz, loss = torch.empty_like(z), torch.empty(3, device=DEV)
    Z.zero_distill_loss(z, 3, 400, ids, t, 6, None, tau, None, 1.0, None, loss, None, dz)

    def value(x):
        Z.zero_distill_loss(x, 3, 400, ids, t, 6, None, tau, None, 1.0, None, loss, None, None)
        return float(loss.double().sum())

    for _ in range(4):
        v = torch.randn(z.shape, generator=g, device=DEV)
        v /= v.norm()
        num = (value(z + step * v) - value(z - step * v)) / (2 * step)
        assert abs(num - float((dz.double() * v.double()).sum())) <= 2e-3


def test_offsets_past_32_bits(Z):
    rows, cols = 17000, 128256                     # 2.2e9 logits
    z = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    _, zl, idl, tl = problem(14, 2, cols, 8, BF16)
    z[-2:] = zl
    ids, t = idl[-1:].expand(rows, 8).contiguous(), tl[-1:].expand(rows, 8).contiguous()
    ids[-2:], t[-2:] = idl, tl
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dz = torch.empty_like(z)
    Z.zero_distill_loss(z, rows, cols, ids, t, 8, None, 1.0, None, 1.0, None, loss, lse, dz)
    check(z[-3:], ids[-3:], t[-3:], 1.0, None, 1.0, loss[-3:], lse[-3:], dz[-3:])


def test_another_stream_and_the_same_bits(Z):
    _, z, ids, t = problem(15, 50, 50257, 20, F16)
    s = torch.cuda.Stream()
    outs = []
    for stream in (torch.cuda.current_stream(), s, s):
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            loss, lse, dz = torch.empty(50, device=DEV), torch.empty(50, device=DEV), torch.empty_like(z)
            Z.zero_distill_loss(z * 2, 50, 50257, ids, t, 20, None, 1.0, None, 1.0, None, loss, lse, dz)
        stream.synchronize()
        outs.append((loss, lse, dz))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], o))


@pytest.mark.parametrize("rows", [1, 5, 50000])
def test_rows_of_no_columns(Z, rows):
    """No id is a column: every row is without entries, and its log-sum-exp is that of nothing."""
    z, k = torch.empty(rows, 0, dtype=BF16, device=DEV), 3
    ids, t = torch.zeros(rows, k, dtype=torch.int64, device=DEV), torch.ones(rows, k, device=DEV)
    loss, lse = (torch.full((rows + 1,), 7.0, device=DEV) for _ in range(2))
    Z.zero_distill_loss(z, rows, 0, ids, t, k, None, 1.0, None, 1.0, None, loss, None, z)
    assert not loss[:rows].any() and loss[rows] == 7 and bool((lse == 7).all())
    loss.fill_(7.0)
    Z.zero_distill_loss(z, rows, 0, ids, t, k, None, 1.0, None, 1.0, None, loss, lse, None)
    assert not loss[:rows].any() and loss[rows] == 7
    assert bool((lse[:rows] == -math.inf).all()) and lse[rows] == 7
    Z.zero_distill_backward(z, rows, 0, ids, t, k, None, 1.0, None, 1.0, None, lse, z)
    Z.zero_distill_loss(z[:0], 0, 0, ids[:0], t[:0], k, None, 1.0, None, 1.0, None, loss[:0], lse[:0], None)


@pytest.mark.parametrize("off", [1e4, -1e4, 1e6])
@pytest.mark.parametrize("tau", [1.0, 3.0])
def test_a_teacher_far_from_zero(Z, off, tau):
    """Only differences of the teacher's logits count: p is as near as that of logits about 0."""
    g, z, ids, t = problem(16, 9, 3000, 70, F32)
    t += off
    loss, lse, dz = torch.empty(9, device=DEV), torch.empty(9, device=DEV), torch.empty_like(z)
    Z.zero_distill_loss(z, 9, 3000, ids, t, 70, None, tau, None, 1.0, None, loss, lse, dz)
    check(z, ids, t, tau, None, 1.0, loss, lse, dz)
    Z.zero_distill_backward(z, 9, 3000, ids, t, 70, None, tau, None, 1.0, None, lse, dz)
    check(z, ids, t, tau, None, 1.0, None, None, dz)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0])
def test_a_teacher_of_the_lowest_values(Z, dtype, tau):
    """Entries masked with the type's lowest value count for nothing beside others, and alike among themselves; the
    same of its largest value.  The reference is given the teacher's logits less their largest: 64 bits do not hold
    3e38 + log 600."""
    low, k = torch.finfo(dtype).min, 600
    _, z, ids, t = problem(17, 6, 3000, k, dtype)
    t[0, 1:], t[1], t[2, 300:] = low, low, low
    t[3, 7], t[3, 500], t[4] = -low, -low, low / 1.5
    near = t.double() - t.double().amax(1, keepdim=True)
    loss, dz = torch.empty(6, device=DEV), torch.empty_like(z)
    Z.zero_distill_loss(z, 6, 3000, ids, t, k, None, tau, None, 1.0, None, loss, None, dz)
    check(z, ids, near, tau, None, 1.0, loss, None, dz)
    lse = torch.logsumexp(z.double() / tau, 1).float()
    Z.zero_distill_backward(z, 6, 3000, ids, t, k, None, tau, None, 1.0, None, lse, dz)
    check(z, ids, near, tau, None, 1.0, None, None, dz)
    t[3, 7], t[3, 500] = 1.0, 1.0
    t_lse = torch.logsumexp(t.double() / tau, 1).float()
    t_lse = torch.where(t_lse > -1e4, t_lse + 0.3, 0.0)            # beside the rest of the teacher's vocabulary
    Z.zero_distill_loss(z, 6, 3000, ids, t, k, t_lse, tau, None, 1.0, None, loss, None, dz)
    check(z, ids, t, tau, None, 1.0, loss, None, dz, t_lse)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("tau", [0.25, 1.0, 2.0])
@pytest.mark.parametrize("cols", [3000, 70001])
@pytest.mark.parametrize("copies", [1, 50])
def test_logits_of_the_lowest_values(Z, dtype, tau, cols, copies):
    """A row masked with the type's lowest value throughout is a uniform one, and any row of finite logits has a
    finite gradient.  The reference is given the logits less their largest (64 bits do not hold 3e38 + log cols);
    losses are compared where fp32 holds log q of every entry."""
    low, k, rows = torch.finfo(dtype).min, 40, 8 * copies
    g, z, ids, t = problem(18, 8, cols, k, dtype)
    z[0], z[1] = low, low
    z[1, 77] = 2.0
    z[2, :cols // 2], z[2, cols // 2:] = low, low / 1.5
    z[3] = -low
    z[4] = torch.where(torch.rand(cols, generator=g, device=DEV) < 0.5, low / 64, -low / 64)
    if dtype != F16:
        z[5], z[6] = (z[5].float() * 1e4 + 1e10).to(dtype), (z[6].float() * 100 - 5e8).to(dtype)
    z[7, cols // 3:] = low                                         # a part of the vocabulary
    z, ids, t = (x.repeat(copies, 1) for x in (z, ids, t))
    loss, lse, dz = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), z.clone()
    Z.zero_distill_loss(dz, rows, cols, ids, t, k, None, tau, None, 1.0, None, loss, lse, dz)
    top = z.double().amax(1, keepdim=True)
    rl, rlse, rdz, mag, size = reference(z.double() - top, ids, t, tau, None, 1.0)
    full = top[:, 0] / tau + rlse
    # at a temperature below 1 the lowest value's lse is itself beyond fp32, and rounds to infinity
    near = (lse.double() - full).abs() <= 2.0 ** -20 + full.abs() * 2.0 ** -23
    assert bool((near | (lse == full.float())).all())
    lim = rdz.abs() * U[dtype] + mag * 2.0 ** -17 + (2.0 ** -25 if dtype == F16 else 1e-37)
    assert bool(((dz.double() - rdz).abs() <= lim).all())
    holds = [r for r in range(rows) if r % 8 not in (1, 2, 7)] if dtype != F16 else range(rows)
    lim = 2.0 ** -19 * tau * tau * (1 + size + full.abs())
    assert bool(((loss.double() - rl).abs() <= lim)[list(holds)].all())

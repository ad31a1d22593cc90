"""zero_layernorm_forward / zero_layernorm_backward at the shapes that training
gives them: several rows under way in a block, four units a lane, rows whose
weights lie packed in shared memory, and rounds in which only some of a block's
groups have a row.  Formulas and tolerances are test_gpu_layernorm.py's; the
restated rule of the launches (layernorm_rule.py) says that the sizes reach
every kernel there is."""
import pytest
import torch

import block_helpers as B
import layernorm_rule as R
import test_gpu_layernorm as T

NAMES = {T.F16: "f16", T.BF16: "bf16", T.F32: "f32"}
TYPES = [(T.F16, T.F16), (T.BF16, T.BF16), (T.F32, T.F32), (T.F16, T.F32), (T.BF16, T.F32)]
# 1300 and 2500 rows: the last round of 152 blocks of 8, 5, 4 or 3 groups is a part of one
SIZES = [(1300, 1600), (2500, 1600), (700, 3456), (1300, 1337), (500, 4097), (3, 8200), (3, 9200), (3, 12288), (3, 14336)]


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


def reached(sizes, backward, sms=152):
    """(rows, cols) of `sizes` by the kernel that they reach: {template: [(groups, blocks, rule, rows)]}."""
    found = {}
    for rows, cols in sizes:
        for xt, rt in TYPES:
            for off in (0, 1):
                k, g, blocks, rule = R.kernel(backward, rows, cols, NAMES[xt], NAMES[rt], NAMES[xt], not off and cols % 8 == 0, sms)
                found.setdefault(k, []).append((g, blocks, rule, rows))
    return found


def every_kernel(backward):
    way = "backward" if backward else "forward"
    for xt, rt in TYPES:
        x, r = NAMES[xt], NAMES[rt]
        for shift in (False, True):
            yield way, x, r, 2, False, shift
            yield way, x, r, "long", False, shift
            # a backward pass of fp32 rows never takes four units a lane: shared memory holds more threads of two
            if not (backward and x == "f32"):
                yield way, x, r, 4, False, shift
            if x != "f32":
                yield way, x, r, 4, True, shift


@pytest.mark.parametrize("backward", [0, 1])
def test_the_sizes_reach_every_kernel(backward):
    found = reached(T.SIZES + SIZES, backward)
    assert set(found) == set(every_kernel(backward))
    for way, x, r, nv, packed, shift in found:
        calls = found[way, x, r, nv, packed, shift]
        groups = max(c[0] for c in calls)
        # several groups a block, and a last round that not all of them have a row in, where any shape has several groups
        part = any(g > 1 and rows % (g * blocks) > 0 and rows > g * blocks for g, blocks, _, rows in calls)
        if nv == 4 and not packed and not (backward and r == "f32"):
            assert groups > 1 or x == "f32"
            if not backward and x != "f32":
                assert groups == 8 and part
            if backward:
                assert groups >= (3 if shift else 8)
    if backward:
        assert any(rule == "two for their threads" for calls in found.values() for _, _, rule, _ in calls)


@pytest.mark.parametrize("backward", [0, 1])
def test_four_units_of_fp32_rows(backward):
    """What no shape would take: a backward pass of fp32 rows with four units a lane, whatever its rows and columns."""
    four = {(rows, cols) for rows in (1, 153, 400, 1300, 9000) for cols in range(1, 20001, 8)
            if R.kernel(backward, rows, cols, "f32", "f32", "f32", cols % 8 == 0, 152)[0][3] == 4}
    assert bool(four) == (not backward)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_forward_and_backward(Z, rows, cols, xt, rt, off, p):
    T.test_forward_and_backward(Z, rows, cols, xt, rt, off, p)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1300, 1600), (3, 14336), (1300, 1337)])
def test_weights_of_another_type(Z, rows, cols):
    """fp32 weights beside 16-bit rows: rows that packed weights would fit are walked instead."""
    g = T.gen(rows + cols)
    x, dy = T.rnd(g, rows, cols, dtype=T.BF16), T.rnd(g, rows, cols, dtype=T.BF16)
    w, b = T.rnd(g, cols, mean=1.0), T.rnd(g, cols)
    y, dr, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=T.DEV), torch.empty(rows, device=T.DEV)
    Z.zero_layernorm_forward(x, None, None, w, b, rows, cols, T.EPS, None, y, mean, rstd)
    ref = T.Ref(x, w, b)
    ref.check_forward(y, mean, rstd)
    dw, db, ws = torch.empty_like(w), torch.empty_like(b), T.workspace(Z, cols)
    Z.zero_layernorm_backward(dy, x, w, rows, cols, mean, rstd, None, None, dr, None, dw, db, 0, ws, ws.numel())
    ref.check_backward(dy, None, dr, None, dw, db)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1300, 1600), (1300, 1337), (700, 3456), (500, 4097)])
def test_sums_added_and_the_same_bits(Z, rows, cols):
    """dw and db added to what a bucket holds, twice with the same bits, dr over dh and dx over dy."""
    g = T.gen(rows - cols)
    h, dy, dh = (T.rnd(g, rows, cols, dtype=T.BF16) for _ in range(3))
    w, drop, k = T.rnd(g, cols, dtype=T.BF16, mean=1.0), Z.drop(0.1, 21, 2, 3), B.keep(rows, cols, 0.1, 21, 2, 3)
    y, mean, rstd = torch.empty_like(h), torch.empty(rows, device=T.DEV), torch.empty(rows, device=T.DEV)
    Z.zero_layernorm_forward(h, None, None, w, None, rows, cols, T.EPS, None, y, mean, rstd)
    ref, old, out = T.Ref(h, w, None), T.rnd(g, 2 * cols), []
    for _ in range(2):
        bucket, dr, dx, ws = old.clone(), dh.clone(), dy.clone(), T.workspace(Z, cols)
        Z.zero_layernorm_backward(dx, h, w, rows, cols, mean, rstd, dr, drop, dr, dx, bucket[:cols], bucket[cols:], 1, ws, ws.numel())
        out.append((bucket, dr, dx))
    assert all(torch.equal(p, q) for p, q in zip(*out))
    ref.check_backward(dy, dh, dr, dx, None, None, k, 0.1)
    _, _, rw, sw, rb, sb = ref.gradients(dy, dh)
    was = old.double()
    T.near(bucket[:cols], was[:cols] + rw, T.F32, (rows + 256) * T.E * (sw + was[:cols].abs()), "dw")
    T.near(bucket[cols:], was[cols:] + rb, T.F32, (rows + 256) * T.E * (sb + was[cols:].abs()), "db")


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1300, 1600), (2500, 333), (700, 8200), (300, 15000), (300, 16384), (300, 16385), (200, 20001), (20, 200000), (3, 1 << 20)])
@pytest.mark.parametrize("dtype", [T.BF16, T.F32])
def test_nothing_behind_the_workspace_is_written(Z, rows, cols, dtype):
    """Sums right and the bytes behind them as they were.  A thread of a walked row adds cols / 512 terms one after the
    other, for the mean and again for the squares: cols / 256 roundings more than test_gpu_layernorm.py counts."""
    g = T.gen(cols)
    h, dy = T.rnd(g, rows, cols, dtype=dtype), T.rnd(g, rows, cols, dtype=dtype)
    y, dr = torch.empty_like(h), torch.empty_like(h)
    mean, rstd = torch.empty(rows, device=T.DEV), torch.empty(rows, device=T.DEV)
    Z.zero_layernorm_forward(h, None, None, None, None, rows, cols, T.EPS, None, y, mean, rstd)
    n = Z.zero_layernorm_workspace_bytes(cols)
    ws = torch.full((n + 4 * cols,), 0x5A, dtype=torch.uint8, device=T.DEV)
    dw, db = torch.empty(cols, device=T.DEV), torch.empty(cols, device=T.DEV)
    Z.zero_layernorm_backward(dy, h, None, rows, cols, mean, rstd, None, None, dr, None, dw, db, 0, ws[:n], n)
    _, _, rw, sw, rb, sb = T.Ref(h, None, None).gradients(dy, None)
    T.near(dw, rw, T.F32, (rows + 256 + cols // 256) * T.E * sw, "dw")
    T.near(db, rb, T.F32, (rows + 256) * T.E * sb, "db")
    assert bool((ws[n:] == 0x5A).all())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(5, 1600), (300, 640), (77, 2568), (77, 2569), (1300, 1600), (3, 14336), (3, 20000), (3, 20001)])
@pytest.mark.parametrize("xt,rt", TYPES)
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("p", [0.1, 0.25])
def test_h_has_the_bits_of_the_fp32_form(Z, rows, cols, xt, rt, off, p):
    """dropout(x) and its sum with the residual each rounded to fp32, as zero_dropout and the elementary operations do."""
    g = T.gen(rows + cols)
    x, r = T.rnd(g, rows, cols, dtype=xt, std=0.5, off=off), T.rnd(g, rows, cols, dtype=rt, std=2.0, mean=0.25, off=off)
    h, y = torch.empty_like(r), torch.empty_like(x)
    Z.zero_layernorm_forward(x, r, Z.drop(p, 13, 5, 7), None, None, rows, cols, T.EPS, h, y, None, None)
    k = B.keep(rows, cols, p, 13, 5, 7)
    product = torch.where(k, x.float() * torch.tensor(B.scale(p), dtype=T.F32, device=T.DEV), torch.zeros((), device=T.DEV))
    want = (product + r.float()).to(rt)
    assert torch.equal(h, want), int((h != want).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,off", [(700, 1600, 0), (700, 1337, 0), (700, 1600, 1), (5, 16400, 0), (5, 16403, 1)])
@pytest.mark.parametrize("dtype", [T.BF16, T.F32])
def test_gradients_over_each_other_s_places(Z, rows, cols, off, dtype):
    """dr over dy with dx over dh, dx alone over dh, dr alone over dy: the bits of outputs of their own."""
    g = T.gen(cols)
    h, dy, dh = (T.rnd(g, rows, cols, dtype=dtype, off=off) for _ in range(3))
    w, drop = T.rnd(g, cols, dtype=dtype, mean=1.0), Z.drop(0.1, 21, 2, 3)
    y, mean, rstd = torch.empty_like(h), torch.empty(rows, device=T.DEV), torch.empty(rows, device=T.DEV)
    Z.zero_layernorm_forward(h, None, None, w, None, rows, cols, T.EPS, None, y, mean, rstd)

    def backward(dy, dh, dr, dx):
        dw, db, ws = torch.empty(cols, device=T.DEV), torch.empty(cols, device=T.DEV), T.workspace(Z, cols)
        Z.zero_layernorm_backward(dy, h, w, rows, cols, mean, rstd, dh, drop, dr, dx, dw, db, 0, ws, ws.numel())
        return dr, dx, dw, db

    new = lambda t: T.rnd(g, rows, cols, dtype=dtype, off=off).copy_(t)
    want = backward(dy, dh, torch.empty_like(h), torch.empty_like(h))
    for over_dy, over_dh in (("dr", "dx"), (None, "dx"), ("dr", None)):
        a, b = new(dy), new(dh)
        got = backward(a, b, a if over_dy else None, b if over_dh else None)
        for p, q in zip(got, want):
            assert p is None or torch.equal(p, q)

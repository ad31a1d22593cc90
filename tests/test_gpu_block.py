"""The block operators together, as a ZeRO-3 unit's training step uses them: the
sublayer's output dropped out onto the residual stream and normed, the gated
block, its second matrix (a plain product here), the way back, the gradients
straight into the ranks' buckets, and the chained partial step, whose chain
gives the dropout its step."""
import math

import pytest
import torch

import block_helpers as B

pytestmark = pytest.mark.gpu
DEV, BF16 = "cuda", torch.bfloat16
U = 2.0 ** -8
ROWS, COLS, FF, RANKS, P, EPS = 200, 256, 704, 2, 0.1, 1e-5


@pytest.fixture(scope="module")
def Z():
    import zero_dp_partitioned_gb300 as Z
    return Z


class Unit:
    """[norm weight | norm bias | gate | up] flat, its second matrix apart and fixed."""

    def __init__(self, Z):
        self.Z = Z
        self.numel = 2 * COLS + 2 * FF * COLS
        g = torch.Generator(device=DEV).manual_seed(0)
        self.params = torch.cat([torch.ones(COLS, device=DEV), torch.zeros(COLS, device=DEV),
                                 torch.randn(2 * FF * COLS, generator=g, device=DEV) * COLS ** -0.5]).to(BF16)
        self.down = (torch.randn(COLS, FF, generator=g, device=DEV) * FF ** -0.5).to(BF16)
        self.state = [torch.empty(self.numel, device=DEV) for _ in range(6)]
        self.buckets = [torch.zeros(self.numel, dtype=BF16, device=DEV) for _ in range(RANKS)]
        n = self.numel // RANKS
        self.shards = [Z.shard(n, r * n, r * n, *(s[r * n:(r + 1) * n] for s in self.state)) for r in range(RANKS)]
        Z.zero_shard_init(self.shards, self.params, Z.ZERO_BF16)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    @staticmethod
    def views(flat):
        return (flat[:COLS], flat[COLS:2 * COLS], flat[2 * COLS:2 * COLS + FF * COLS].view(FF, COLS),
                flat[2 * COLS + FF * COLS:].view(FF, COLS))

    def passes(self, rank, x, residual, dout, chain, out):
        """One rank's forward and backward pass; gradients into its bucket."""
        Z = self.Z
        w, b, wg, wu = self.views(self.params)
        dw, db, dwg, dwu = self.views(self.buckets[rank])
        e = lambda r, c: torch.empty(r, c, dtype=BF16, device=DEV)
        drop = Z.drop(P, 1000 + rank, site=3, chain_dev=chain)
        h, y, mean, rstd = e(ROWS, COLS), e(ROWS, COLS), torch.empty(ROWS, device=DEV), torch.empty(ROWS, device=DEV)
        Z.zero_layernorm_forward(x, residual, drop, w, b, ROWS, COLS, EPS, h, y, mean, rstd)
        act, gate, up = e(ROWS, FF), e(ROWS, FF), e(ROWS, FF)
        Z.zero_gated_forward(y, wg, wu, ROWS, COLS, FF, Z.ZERO_SILU, act, gate, up, None, 0, self.status)
        down = act @ self.down.t()
        # what leaves the unit: the residual stream and the block's output, dropped out onto it
        last = e(ROWS, COLS)
        Z.zero_dropout(down, h, ROWS, COLS, Z.drop(P, 1000 + rank, site=4, chain_dev=chain), last)
        ddown, dx, dr = e(ROWS, COLS), e(ROWS, COLS), e(ROWS, COLS)
        Z.zero_dropout(dout, None, ROWS, COLS, Z.drop(P, 1000 + rank, site=4, chain_dev=chain), ddown)
        dact, dy = ddown @ self.down, e(ROWS, COLS)
        n = Z.zero_gated_backward_workspace_bytes(y, wg, wu, gate, up, ROWS, COLS, FF)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
        Z.zero_gated_backward(dact, gate, up, y, wg, wu, ROWS, COLS, FF, Z.ZERO_SILU, gate, up, dy, dwg, dwu, 0, ws, n, self.status)
        lws = torch.empty(Z.zero_layernorm_workspace_bytes(COLS), dtype=torch.uint8, device=DEV)
        Z.zero_layernorm_backward(dy, h, w, ROWS, COLS, mean, rstd, dout, drop, dr, dx, dw, db, 0, lws, lws.numel())
        out.update(last=last, dx=dx, dr=dr)


def reference(unit, rank, x, residual, dout, step):
    """The same in 64 bits, each stored value rounded as the calls store it."""
    r16 = lambda t: t.to(BF16).double()
    w, b, wg, wu = (t.double() for t in unit.views(unit.params))
    x, residual, dout, wd = x.double(), residual.double(), dout.double(), unit.down.double()
    k1, k2 = (B.keep(ROWS, COLS, P, 1000 + rank, s, step).double() * B.scale(P) for s in (3, 4))
    h = r16(x * k1 + residual)
    m = h.mean(1, keepdim=True)
    rstd = ((h - m).pow(2).mean(1, keepdim=True) + EPS).pow(-0.5)
    xh = (h - m) * rstd
    y = r16(xh * w + b)
    g, u = y @ wg.t(), y @ wu.t()
    act = r16(torch.sigmoid(g) * g * u)
    last = r16(r16(act @ wd.t()) * k2 + h)
    g, u = r16(g), r16(u)
    da = r16(r16(dout * k2) @ wd)
    s = torch.sigmoid(g)
    dg, du = r16(da * u * (s + g * s * (1 - s))), r16(da * g * s)
    dy = r16(dg @ wg + du @ wu)
    gw = dy * w
    dr = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) + dout
    return {"last": last, "dx": dr * k1, "dr": dr}, ((dy * xh).sum(0), dy.sum(0), dg.t() @ y, du.t() @ y)


def close(got, ref, what):
    """Both round the same values, in fp32 and in 64 bits before it: a value in
    some hundred lands on the other side (fp32 sums are within 2^-17, a step is
    2^-7) and is a step (2 U of itself) off, U / 4 of the norm a rounding; sixteen
    roundings, and the last one's U."""
    err = float((got.double() - ref).norm() / ref.norm())
    assert err < 5 * U, (what, err)


def test_a_unit_trains(Z):
    unit = Unit(Z)
    g = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda std: (torch.randn(ROWS, COLS, generator=g, device=DEV) * std).to(BF16)
    hyper = Z.hyper(lr=1e-3, weight_decay=0.0)
    table = torch.from_numpy(Z.zero_adam_scalar_table(hyper, 1, 8)).to(DEV)
    chain = torch.frombuffer(bytearray(bytes(Z.chain(loss_scale=1.0))), dtype=torch.uint8).to(DEV)
    ws = torch.zeros(Z.zero_workspace_bytes(), dtype=torch.uint8, device=DEV)
    stats, result = (torch.zeros(n, dtype=torch.uint8, device=DEV) for n in (16, 48))
    for step in (1, 2, 3):
        bad = step == 2
        before = unit.params.clone()
        for rank in range(RANKS):
            x, residual, dout = rnd(0.5), rnd(2.0), rnd(1e-2)
            if bad and rank == 1:
                dout[7, 9] = math.inf
            out = {}
            unit.passes(rank, x, residual, dout, chain, out)
            if not bad:
                want, grads = reference(unit, rank, x, residual, dout, step if step == 1 else 2)
                for k, v in want.items():
                    close(out[k], v, (step, rank, k))
                for got, ref, k in zip(unit.views(unit.buckets[rank]), grads, ("dw", "db", "dgate_w", "dup_w")):
                    close(got, ref, (step, rank, k))
        Z.zero_shard_step_partial(unit.buckets, Z.ZERO_BF16, unit.shards, unit.params, Z.ZERO_BF16, hyper, 1.0, 0, stats, ws,
                                  ws.numel(), scalar_table=table, table_t0=1, n_table=8, chain_dev=chain)
        Z.zero_shard_step_commit(unit.shards, unit.params, Z.ZERO_BF16, 1.0, stats, 0.0, 0, result, table_t0=1, n_table=8,
                                 chain_dev=chain)
        torch.cuda.synchronize()
        # an infinite gradient reaches the buckets: the step is skipped, t and with it the masks stay
        assert torch.equal(unit.params, before) == bad
    c = Z.read_chain(chain)
    assert (c.applied, c.skipped, c.step) == (2, 1, 3) and int(unit.status) == 0

"""CPU tests of the block operators (layer norm, dropout, gated feed-forward):
each refusal comes before any device work, the host-only sizes, and the
reference generator that the GPU tests take the mask from."""
import ctypes

import pytest
import torch

import block_helpers as B

FAKE = 0x10000      # an aligned address that is never dereferenced: every case fails validation first


@pytest.fixture(scope="module")
def Z():
    import __graft_entry__
    __graft_entry__.build()
    import zero_dp_partitioned_gb300 as Z
    return Z


def refused(Z, code, f, *args):
    with pytest.raises(Z.ZeroError) as e:
        f(*args, stream=0)
    assert e.value.code == code, str(e.value)
    assert str(e.value)


def m(Z, ld=64, dtype=2, data=FAKE):
    return Z.mat(data, ld, dtype)


def test_the_reference_generator_has_the_published_values():
    """The known answers of the generator's authors (Random123)."""
    assert B.philox((0,) * 4, (0,) * 2) == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    assert B.philox((B.LOW,) * 4, (B.LOW,) * 2) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert B.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)


def test_the_reference_mask_is_the_generators():
    rows, cols, p, seed, site, step = 3, 21, 0.3, 0x123456789ABCDEF0, 5, 2 ** 32 + 9
    got = B.keep(rows, cols, p, seed, site, step, device="cpu")
    for r in range(rows):
        for c in range(cols):
            w = B.philox((r * 3 + c // 8, 0, site, 9), (seed & B.LOW, seed >> 32))[c % 8 // 2]
            assert bool(got[r, c]) == ((w >> 16 * (c % 2) & 0xFFFF) >= B.limit(p))
    big = B.keep(2000, 800, 0.1, 1, 2, 3, device="cpu").double().mean()
    # 1.6 million trials: the standard deviation is 2.4e-4
    assert abs(float(big) - (1 - B.limit(0.1) / 65536)) < 1.5e-3


def test_struct_size(Z):
    assert ctypes.sizeof(Z.zero_drop) == 32


def test_dropout_refusals(Z):
    def call(code, **kw):
        a = dict(x=m(Z), residual=m(Z), rows=4, cols=64, drop=Z.drop(0.1, 1), y=m(Z))
        a.update(kw)
        refused(Z, code, Z.zero_dropout, *a.values())

    call(Z.ZERO_EINVAL, rows=-1)
    call(Z.ZERO_EINVAL, cols=-1)
    call(Z.ZERO_ELIMIT, rows=1 << 40, cols=1 << 30)
    call(Z.ZERO_EINVAL, drop=None)
    for p in (-0.1, 1.1, float("nan")):
        call(Z.ZERO_EINVAL, drop=Z.drop(p, 1))
    call(Z.ZERO_EALIGN, drop=Z.drop(0.1, 1, chain_dev=FAKE + 4))
    call(Z.ZERO_EINVAL, x=None)
    call(Z.ZERO_EINVAL, x=m(Z, dtype=4))
    call(Z.ZERO_EINVAL, x=m(Z, ld=63))
    call(Z.ZERO_EALIGN, x=m(Z, data=FAKE + 1))
    call(Z.ZERO_EINVAL, y=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, residual=m(Z, dtype=1))
    call(Z.ZERO_EINVAL, y=m(Z, data=0))
    call(Z.ZERO_EINVAL, x=torch.zeros(4, 63, dtype=torch.bfloat16))
    with pytest.raises(Z.ZeroError):
        Z.drop(0.1, 1, chain_dev=torch.zeros(55, dtype=torch.uint8))
    with pytest.raises(Z.ZeroError):
        Z.drop(0.1, 1, chain_dev=torch.zeros(56, dtype=torch.uint8))       # not on a GPU
    Z.zero_dropout(m(Z), None, 0, 64, Z.drop(0.1, 1), m(Z), stream=0)      # nothing to do, nothing launched
    Z.zero_dropout(m(Z), None, 4, 0, Z.drop(0.1, 1), m(Z), stream=0)


def test_layernorm_forward_refusals(Z):
    def call(code, **kw):
        a = dict(x=m(Z), residual=m(Z), drop=Z.drop(0.1, 1), weight=m(Z), bias=m(Z), rows=4, cols=64, eps=1e-5,
                 h_out=m(Z), y=m(Z), mean=FAKE, rstd=FAKE)
        a.update(kw)
        refused(Z, code, Z.zero_layernorm_forward, *a.values())

    call(Z.ZERO_EINVAL, rows=-1)
    call(Z.ZERO_EINVAL, cols=-1)
    call(Z.ZERO_ELIMIT, cols=(1 << 20) + 1)
    for eps in (-1.0, float("nan"), float("inf")):
        call(Z.ZERO_EINVAL, eps=eps)
    call(Z.ZERO_EINVAL, x=None)
    call(Z.ZERO_EINVAL, x=m(Z, dtype=4))
    call(Z.ZERO_EINVAL, x=m(Z, ld=63))
    call(Z.ZERO_EALIGN, x=m(Z, data=FAKE + 1))
    call(Z.ZERO_EINVAL, residual=m(Z, dtype=1))
    call(Z.ZERO_EINVAL, h_out=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, y=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, y=m(Z, dtype=4))
    call(Z.ZERO_EINVAL, y=None)
    call(Z.ZERO_EALIGN, mean=FAKE + 1)
    call(Z.ZERO_EALIGN, rstd=FAKE + 2)
    for what in ("weight", "bias"):
        call(Z.ZERO_EINVAL, **{what: m(Z, dtype=5)})
        call(Z.ZERO_EALIGN, **{what: m(Z, data=FAKE + 1)})
        call(Z.ZERO_EINVAL, **{what: m(Z, data=0)})          # a unit that is not gathered
    call(Z.ZERO_EINVAL, drop=Z.drop(2.0, 1))
    call(Z.ZERO_EINVAL, mean=torch.zeros(3))


def test_layernorm_backward_refusals(Z):
    ws = Z.zero_layernorm_workspace_bytes(64)
    assert ws >= 2 * 64 * 4 and Z.zero_layernorm_workspace_bytes(0) == 0

    def call(code, **kw):
        a = dict(dy=m(Z), h=m(Z), weight=m(Z), rows=4, cols=64, mean=FAKE, rstd=FAKE, dh=m(Z), drop=Z.drop(0.1, 1),
                 dr=m(Z), dx=m(Z), dw=m(Z), db=m(Z), accumulate=0, workspace=FAKE, workspace_bytes=ws)
        a.update(kw)
        refused(Z, code, Z.zero_layernorm_backward, *a.values())

    call(Z.ZERO_EINVAL, rows=-1)
    call(Z.ZERO_EINVAL, dy=None)
    call(Z.ZERO_EINVAL, h=m(Z, dtype=1))
    call(Z.ZERO_EINVAL, mean=None)
    call(Z.ZERO_EINVAL, rstd=FAKE + 1)
    call(Z.ZERO_EINVAL, dr=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, dx=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, dr=None, dx=None)
    call(Z.ZERO_EINVAL, dh=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, dw=m(Z, dtype=4))
    call(Z.ZERO_EALIGN, db=m(Z, data=FAKE + 1))
    call(Z.ZERO_EINVAL, weight=m(Z, data=0))
    call(Z.ZERO_EWORKSPACE, workspace=None)
    call(Z.ZERO_EWORKSPACE, workspace_bytes=ws - 1)
    call(Z.ZERO_EWORKSPACE, dw=None, workspace_bytes=ws - 1)
    call(Z.ZERO_EWORKSPACE, workspace=torch.zeros(ws - 1, dtype=torch.uint8))
    call(Z.ZERO_ELIMIT, cols=(1 << 20) + 1)
    call(Z.ZERO_EINVAL, drop=Z.drop(-1.0, 1))


def test_gated_forward_refusals(Z):
    def call(code, **kw):
        a = dict(x=m(Z), gate_w=m(Z), up_w=m(Z), rows=9, cols=64, ff=64, act=0, h=m(Z), gate=m(Z), up=m(Z),
                 workspace=None, workspace_bytes=0, status=FAKE)
        a.update(kw)
        refused(Z, code, Z.zero_gated_forward, *a.values())

    for size in ("rows", "cols", "ff"):
        call(Z.ZERO_EINVAL, **{size: -1})
        call(Z.ZERO_ELIMIT, **{size: 1 << 31})
    call(Z.ZERO_ELIMIT, rows=1 << 29, ff=1 << 29)                # too many tiles
    call(Z.ZERO_EINVAL, act=2)
    call(Z.ZERO_EINVAL, act=-1)
    for what in ("x", "gate_w", "up_w", "h"):
        call(Z.ZERO_EINVAL, **{what: None})
    for what in ("x", "gate_w", "up_w", "h", "gate", "up"):
        call(Z.ZERO_EINVAL, **{what: m(Z, data=0)})
        call(Z.ZERO_EINVAL, **{what: m(Z, dtype=3)})
        call(Z.ZERO_EINVAL, **{what: m(Z, dtype=1)})             # fp16 beside bf16
        call(Z.ZERO_EINVAL, **{what: m(Z, ld=63)})
        call(Z.ZERO_EALIGN, **{what: m(Z, data=FAKE + 1)})
    call(Z.ZERO_EINVAL, gate=None)
    call(Z.ZERO_EINVAL, up=None)
    call(Z.ZERO_EINVAL, status=None)
    call(Z.ZERO_EINVAL, status=FAKE + 2)
    call(Z.ZERO_EWORKSPACE, x=m(Z, data=FAKE + 2))               # rows off 16 bytes need a copy
    need = Z.zero_gated_forward_workspace_bytes(m(Z), m(Z, ld=65), m(Z), 9, 64, 64)
    assert need == 64 * 64 * 2
    assert Z.zero_gated_forward_workspace_bytes(m(Z), m(Z, ld=65), m(Z), 4, 64, 64) == 0      # few rows: read where they lie
    call(Z.ZERO_EWORKSPACE, gate_w=m(Z, ld=65), workspace=FAKE, workspace_bytes=need - 1)
    call(Z.ZERO_EWORKSPACE, gate_w=m(Z, ld=65), workspace=FAKE + 8, workspace_bytes=need)
    call(Z.ZERO_EINVAL, x=torch.zeros(9, 63, dtype=torch.bfloat16))


def test_gated_backward_refusals(Z):
    def call(code, **kw):
        a = dict(dh=m(Z), gate=m(Z), up=m(Z), x=m(Z), gate_w=m(Z), up_w=m(Z), rows=4, cols=64, ff=64, act=1, dgate=m(Z),
                 dup=m(Z), dx=m(Z), dgate_w=m(Z), dup_w=m(Z), accumulate=0, workspace=None, workspace_bytes=0, status=FAKE)
        a.update(kw)
        refused(Z, code, Z.zero_gated_backward, *a.values())

    for size in ("rows", "cols", "ff"):
        call(Z.ZERO_EINVAL, **{size: -1})
        call(Z.ZERO_ELIMIT, **{size: 1 << 31})
    call(Z.ZERO_EINVAL, act=7)
    for what in ("dh", "gate", "up", "x", "gate_w", "up_w", "dgate", "dup"):
        call(Z.ZERO_EINVAL, **{what: None})
    for what in ("dh", "gate", "up", "x", "gate_w", "up_w", "dgate", "dup", "dx"):
        call(Z.ZERO_EINVAL, **{what: m(Z, dtype=3)})
        call(Z.ZERO_EINVAL, **{what: m(Z, dtype=1)})
        call(Z.ZERO_EALIGN, **{what: m(Z, data=FAKE + 1)})
    call(Z.ZERO_EINVAL, dgate_w=None)
    call(Z.ZERO_EINVAL, dup_w=None)
    call(Z.ZERO_EINVAL, dup_w=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, dgate_w=m(Z, dtype=1), dup_w=m(Z, dtype=1))
    call(Z.ZERO_EINVAL, status=None)
    call(Z.ZERO_EWORKSPACE, dgate=m(Z, ld=65))
    assert Z.zero_gated_backward_workspace_bytes(None, None, None, m(Z), m(Z, ld=70), 4, 64, 100) == 4 * 128 * 2
    assert Z.zero_gated_backward_workspace_bytes(m(Z), m(Z), m(Z), m(Z), m(Z), 4, 64, 64) == 0


def test_the_layernorm_workspace_holds_what_a_launch_writes(Z):
    """A partial dw and db of each of 152 blocks at most; rows that are walked have the few shares of them that fill the GPU."""
    for cols in (1, 1600, 4097, 16384):
        assert Z.zero_layernorm_workspace_bytes(cols) == 152 * cols * 8
    for cols in (16385, 20000, 200000, 1 << 20):
        shares = -(-8 * 152 // -(-cols // 128))
        assert Z.zero_layernorm_workspace_bytes(cols) == shares * cols * 8
    assert Z.zero_layernorm_workspace_bytes((1 << 20) + 1) == 0

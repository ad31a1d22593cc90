"""CPU tests of the layer operators' argument checks: each refusal comes before
any device work (no GPU is touched here), and the host-only sizes."""
import ctypes

import pytest
import torch

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


def test_struct_sizes(Z):
    assert ctypes.sizeof(Z.zero_mat) == 24 and ctypes.sizeof(Z.zero_mx4) == 48


def test_norm_forward_refusals(Z):
    def call(code, **kw):
        a = dict(x=m(Z), residual=m(Z), weight=m(Z), rows=4, cols=64, eps=1e-5, h_out=m(Z), y=m(Z), y_scale=None,
                 scale_block=0, rstd=FAKE)
        a.update(kw)
        refused(Z, code, Z.zero_norm_forward, *a.values())

    call(Z.ZERO_EINVAL, rows=-1)
    call(Z.ZERO_EINVAL, cols=-1)
    call(Z.ZERO_ELIMIT, cols=(1 << 20) + 1)
    for eps in (-1.0, float("nan"), float("inf")):
        call(Z.ZERO_EINVAL, eps=eps)
    call(Z.ZERO_EINVAL, x=None)
    call(Z.ZERO_EINVAL, x=m(Z, data=0))
    call(Z.ZERO_EINVAL, x=m(Z, dtype=4))
    call(Z.ZERO_EINVAL, x=m(Z, dtype=99))
    call(Z.ZERO_EINVAL, x=m(Z, dtype=-1))
    call(Z.ZERO_EINVAL, x=m(Z, ld=63))
    call(Z.ZERO_EALIGN, x=m(Z, data=FAKE + 1))
    call(Z.ZERO_EINVAL, residual=m(Z, dtype=1))              # fp16 beside bf16
    call(Z.ZERO_EINVAL, h_out=m(Z, dtype=3))                 # not the residual's type
    call(Z.ZERO_EINVAL, y=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, y=None)
    call(Z.ZERO_EINVAL, y=m(Z, dtype=4))                     # no y_scale
    call(Z.ZERO_EINVAL, y=m(Z, dtype=4), y_scale=FAKE, scale_block=64)
    call(Z.ZERO_EALIGN, y=m(Z, dtype=4), y_scale=FAKE + 2)
    call(Z.ZERO_EALIGN, rstd=FAKE + 1)
    call(Z.ZERO_EINVAL, weight=m(Z, dtype=5))
    call(Z.ZERO_EALIGN, weight=m(Z, data=FAKE + 1))
    call(Z.ZERO_EINVAL, x=torch.zeros(4, 63, dtype=torch.bfloat16))          # another shape
    call(Z.ZERO_EINVAL, x=torch.zeros(64, 4, dtype=torch.bfloat16).t())      # columns apart
    call(Z.ZERO_EINVAL, rstd=torch.zeros(3))
    call(Z.ZERO_EINVAL, weight=torch.zeros(64, dtype=torch.float64))


def test_norm_backward_refusals(Z):
    ws = Z.zero_norm_workspace_bytes(64)
    assert ws >= 64 * 4 and Z.zero_norm_workspace_bytes(0) == 0

    def call(code, **kw):
        a = dict(dy=m(Z), h=m(Z), weight=m(Z), rows=4, cols=64, rstd=FAKE, dh=m(Z), dx=m(Z), dw=m(Z), accumulate=0,
                 workspace=FAKE, workspace_bytes=ws)
        a.update(kw)
        refused(Z, code, Z.zero_norm_backward, *a.values())

    call(Z.ZERO_EINVAL, rows=-1)
    call(Z.ZERO_EINVAL, dy=None)
    call(Z.ZERO_EINVAL, rstd=None)
    call(Z.ZERO_EINVAL, h=m(Z, dtype=1))
    call(Z.ZERO_EINVAL, dx=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, dh=m(Z, dtype=3))
    call(Z.ZERO_EINVAL, dw=m(Z, dtype=4))
    call(Z.ZERO_EALIGN, dw=m(Z, data=FAKE + 1))
    call(Z.ZERO_EWORKSPACE, workspace=None)
    call(Z.ZERO_EWORKSPACE, workspace_bytes=ws - 1)
    call(Z.ZERO_ELIMIT, cols=(1 << 20) + 1)


def test_distill_refusals(Z):
    def call(code, f=None, **kw):
        a = dict(logits=m(Z), rows=4, cols=64, ids=m(Z, 8, 6), teacher=m(Z, 8), k=8, teacher_lse=None, temperature=1.0,
                 row_weight=None, grad_scale=1.0, chain_dev=None, loss=FAKE, lse=FAKE, dlogits=m(Z))
        a.update(kw)
        refused(Z, code, Z.zero_distill_loss, *a.values())
        del a["loss"]
        if kw.get("loss") is None:
            refused(Z, code, Z.zero_distill_backward, *a.values())

    call(Z.ZERO_EINVAL, rows=-1)
    call(Z.ZERO_EINVAL, cols=-1)
    call(Z.ZERO_EINVAL, k=-1)
    call(Z.ZERO_ELIMIT, k=1025)
    call(Z.ZERO_ELIMIT, cols=1 << 31)
    for t in (0.0, -1.0, float("nan"), float("inf")):
        call(Z.ZERO_EINVAL, temperature=t)
    call(Z.ZERO_EINVAL, grad_scale=float("inf"))
    call(Z.ZERO_EINVAL, logits=m(Z, dtype=4))
    call(Z.ZERO_EINVAL, ids=m(Z, 8, 2))
    call(Z.ZERO_EALIGN, ids=m(Z, 8, 6, FAKE + 4))
    call(Z.ZERO_EINVAL, ids=m(Z, 7, 6))
    call(Z.ZERO_EINVAL, teacher=None)
    call(Z.ZERO_EINVAL, dlogits=m(Z, dtype=3))
    call(Z.ZERO_EALIGN, row_weight=FAKE + 2)
    call(Z.ZERO_EALIGN, chain_dev=FAKE + 4)
    call(Z.ZERO_EALIGN, loss=FAKE + 1)
    call(Z.ZERO_EALIGN, lse=FAKE + 1)
    call(Z.ZERO_EINVAL, row_weight=torch.zeros(3))
    args = (m(Z), 4, 64, m(Z, 8, 6), m(Z, 8), 8, None, 1.0, None, 1.0, None)
    refused(Z, Z.ZERO_EINVAL, Z.zero_distill_backward, *args, None, m(Z))            # no lse
    refused(Z, Z.ZERO_EINVAL, Z.zero_distill_backward, *args, FAKE, None)            # no dlogits


def test_mx4_sizes(Z):
    assert Z.zero_mx4_bytes(1, 1, Z.ZERO_MX4_ROWS) == (16, 16, 1)
    assert Z.zero_mx4_bytes(1, 1) == (16, 16, 1024)
    assert Z.zero_mx4_bytes(129, 257) == (144, 129 * 144, 2 * 2 * 1024)
    assert Z.zero_mx4_bytes(14336, 4096) == (2048, 14336 * 2048, 14336 * 128)
    assert Z.zero_mx4_bytes(14336, 4096, Z.ZERO_MX4_ROWS) == (2048, 14336 * 2048, 14336 * 128)
    assert Z.zero_mx4_bytes(0, 5) == (16, 0, 0)
    for bad in ((-1, 4, 0), (4, -1, 1), (4, 4, 2)):
        with pytest.raises(Z.ZeroError):
            Z.zero_mx4_bytes(*bad)
    q = Z.mx4(3, 70, device="cpu")
    assert (q.rows, q.cols, q.ld) == (3, 70, 48) and q.scales == q.data + 3 * 48
    with pytest.raises(Z.ZeroError):
        Z.mx4(3, 70, torch.zeros(3 * 48 - 1, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8))


def test_mx4_refusals(Z):
    def q(rows=4, cols=64, ld=32, data=FAKE, scales=FAKE, layout=1):
        return Z.zero_mx4(data, scales, rows, cols, ld, layout, 0)

    f = Z.zero_mx4_quantize
    refused(Z, Z.ZERO_EINVAL, f, m(Z), -1, 64, q(), None)
    refused(Z, Z.ZERO_EINVAL, f, m(Z, dtype=4), 4, 64, q(), None)
    refused(Z, Z.ZERO_EINVAL, f, m(Z), 4, 64, q(rows=5), None)
    refused(Z, Z.ZERO_EINVAL, f, m(Z), 4, 64, None, q())                  # the transpose is 64 x 4
    refused(Z, Z.ZERO_EINVAL, f, m(Z), 4, 64, q(ld=16), None)
    refused(Z, Z.ZERO_EINVAL, f, m(Z), 4, 64, q(ld=40), None)
    refused(Z, Z.ZERO_EALIGN, f, m(Z), 4, 64, q(data=FAKE + 8), None)
    refused(Z, Z.ZERO_EALIGN, f, m(Z), 4, 64, q(scales=FAKE + 4), None)
    refused(Z, Z.ZERO_EINVAL, f, m(Z), 4, 64, q(scales=0), None)
    refused(Z, Z.ZERO_EINVAL, f, m(Z), 4, 64, q(layout=2), None)
    refused(Z, Z.ZERO_EINVAL, Z.zero_mx4_dequantize, None, m(Z))
    refused(Z, Z.ZERO_EINVAL, Z.zero_mx4_dequantize, q(), m(Z, dtype=6))
    refused(Z, Z.ZERO_EINVAL, Z.zero_mx4_dequantize, q(), m(Z, ld=63))
    t = Z.zero_mx4_tile_scales
    refused(Z, Z.ZERO_EINVAL, t, q(), q())
    refused(Z, Z.ZERO_EINVAL, t, q(layout=0), q(rows=5))
    mm = Z.zero_mx4_matmul
    refused(Z, Z.ZERO_EINVAL, mm, q(), q(cols=32), 1.0, m(Z), FAKE)
    refused(Z, Z.ZERO_EINVAL, mm, q(layout=0), q(), 1.0, m(Z), FAKE)
    refused(Z, Z.ZERO_EINVAL, mm, q(), q(), 1.0, m(Z, ld=3), FAKE)
    refused(Z, Z.ZERO_EINVAL, mm, q(), q(), 1.0, m(Z, dtype=4), FAKE)
    refused(Z, Z.ZERO_EINVAL, mm, q(), q(), 1.0, m(Z), None)
    refused(Z, Z.ZERO_EINVAL, mm, q(), q(), 1.0, m(Z), FAKE + 2)
    refused(Z, Z.ZERO_EINVAL, mm, q(), q(), float("nan"), m(Z), FAKE)
    refused(Z, Z.ZERO_ELIMIT, mm, q(rows=1 << 31), q(), 1.0, m(Z), FAKE)
    Z.zero_mx4_matmul(q(rows=0), q(), 1.0, m(Z), FAKE, stream=0)          # nothing to do: no launch


def test_buffers_that_are_not_on_a_gpu_are_refused(Z):
    """Matrices, workspace, chain and status given as CPU tensors: an error before any launch."""
    host, n = torch.zeros(4, 64, dtype=torch.bfloat16), Z.zero_norm_workspace_bytes(64)
    u8 = torch.zeros(4096, dtype=torch.uint8)
    q = Z.mx4(4, 64, device="cpu")
    over = Z.mx4(4, 64, u8, FAKE)                                         # one buffer on the host is enough
    gpu = Z.zero_mx4(FAKE, FAKE, 4, 64, 32, 1, 0)
    rows = Z.zero_mx4(FAKE, FAKE, 4, 64, 32, 0, 0)
    e = Z.ZERO_EINVAL
    for bad in (q, over):
        refused(Z, e, Z.zero_mx4_quantize, m(Z), 4, 64, bad, None)
        refused(Z, e, Z.zero_mx4_dequantize, bad, m(Z))
        refused(Z, e, Z.zero_mx4_tile_scales, rows, bad)
        refused(Z, e, Z.zero_mx4_matmul, bad, gpu, 1.0, m(Z), FAKE)
        refused(Z, e, Z.zero_mx4_matmul, gpu, bad, 1.0, m(Z), FAKE)
    refused(Z, e, Z.zero_mx4_quantize, m(Z), 64, 4, None, Z.mx4(4, 64, device="cpu"))
    refused(Z, e, Z.zero_mx4_quantize, Z.mat(host), 4, 64, gpu, None)
    refused(Z, e, Z.zero_mx4_matmul, gpu, gpu, 1.0, m(Z), torch.zeros(1, dtype=torch.int32))
    refused(Z, e, Z.zero_norm_backward, m(Z), m(Z), None, 4, 64, FAKE, None, m(Z), m(Z), 0,
            torch.zeros(n, dtype=torch.uint8), n)
    args = (m(Z), 4, 64, m(Z, 8, 6), m(Z, 8), 8, None, 1.0, None, 1.0, torch.zeros(56, dtype=torch.uint8))
    refused(Z, e, Z.zero_distill_loss, *args, FAKE, FAKE, None)
    refused(Z, e, Z.zero_distill_backward, *args, FAKE, m(Z))


def test_buffers_that_are_too_small_are_refused(Z):
    n = Z.zero_norm_workspace_bytes(64)
    refused(Z, Z.ZERO_EWORKSPACE, Z.zero_norm_backward, m(Z), m(Z), None, 4, 64, FAKE, None, m(Z), m(Z), 0,
            torch.zeros(n - 1, dtype=torch.uint8), n)
    gpu = Z.zero_mx4(FAKE, FAKE, 4, 64, 32, 1, 0)
    refused(Z, Z.ZERO_EINVAL, Z.zero_mx4_matmul, gpu, gpu, 1.0, m(Z), torch.zeros(2, dtype=torch.uint8))
    refused(Z, Z.ZERO_EINVAL, Z.zero_distill_loss, m(Z), 4, 64, m(Z, 8, 6), m(Z, 8), 8, None, 1.0, None, 1.0,
            torch.zeros(55, dtype=torch.uint8), FAKE, FAKE, None)


def test_a_4_bit_matrix_is_made_on_the_current_gpu(Z, monkeypatch):
    where = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: where.append(str(device)) or empty(*a, **k))
    Z.mx4(4, 64)
    assert where == ["cuda"]


def test_the_current_stream_without_torchs_private_calls(Z, monkeypatch):
    """A torch that has renamed them gives the stream by its public calls."""
    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(Z, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: type("S", (), {"cuda_stream": 0x1000 + d}))
    assert Z._stream(None) == 0x1003


class OnGpu:
    """What the calls ask of a tensor, on the GPU of the given number."""

    def __init__(self, gpu, *shape, dtype=torch.bfloat16):
        self.like, self.gpu = torch.empty(*shape, dtype=dtype), gpu
        self.dtype, self.shape, self.is_cuda = dtype, self.like.shape, True

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return FAKE

    def __getattr__(self, name):
        return getattr(self.like, name)


def test_tensors_of_another_gpu_are_refused(Z, monkeypatch):
    """Their addresses mean nothing, or something else, to a kernel on the current one."""
    monkeypatch.setattr(Z, "_raw_stream", (lambda d: 0, lambda: 1))
    monkeypatch.setattr(Z, "_gpus", 2)
    e, f32, u8 = Z.ZERO_EINVAL, torch.float32, torch.uint8
    there = OnGpu(0, 4, 64)
    n = Z.zero_norm_workspace_bytes(64)
    gpu = Z.zero_mx4(FAKE, FAKE, 4, 64, 32, 1, 0)
    refused(Z, e, Z.zero_norm_forward, there, None, None, 4, 64, 1e-5, None, m(Z), None, 0, None)
    refused(Z, e, Z.zero_norm_forward, Z.mat(there), None, None, 4, 64, 1e-5, None, m(Z), None, 0, None)
    refused(Z, e, Z.zero_norm_forward, m(Z), None, None, 4, 64, 1e-5, None, m(Z), None, 0, OnGpu(0, 4, dtype=f32))
    refused(Z, e, Z.zero_norm_backward, m(Z), m(Z), None, 4, 64, FAKE, None, m(Z), m(Z), 0, OnGpu(0, n, dtype=u8), n)
    refused(Z, e, Z.zero_mx4_quantize, m(Z), 4, 64, Z.mx4(4, 64, OnGpu(0, 4096, dtype=u8), FAKE), None)
    refused(Z, e, Z.zero_mx4_matmul, gpu, gpu, 1.0, m(Z), OnGpu(0, 1, dtype=torch.int32))
    with pytest.raises(Z.ZeroError):
        Z.mx4(4, 64, OnGpu(0, 4096, dtype=u8), OnGpu(1, 4096, dtype=u8))
    # on the current one they pass: nothing to do, so nothing is launched
    here = OnGpu(1, 0, 64)
    Z.zero_norm_forward(here, None, None, 0, 64, 1e-5, None, here, None, 0, OnGpu(1, 0, dtype=f32), stream=0)
    Z.zero_mx4_quantize(here, 0, 64, Z.mx4(0, 64, OnGpu(1, 0, dtype=u8), OnGpu(1, 0, dtype=u8)), None, stream=0)


def test_a_weight_without_data_is_refused(Z):
    """An address of 0 (a unit that is not gathered) is not a weight of 1."""
    ws = Z.zero_norm_workspace_bytes(64)
    for dtype in (1, 2, 3):
        w = m(Z, dtype=dtype, data=0)
        for call, f, args in (("zero_norm_forward", Z.zero_norm_forward,
                               (m(Z), None, w, 4, 64, 1e-5, None, m(Z), None, 0, None)),
                              ("zero_norm_backward", Z.zero_norm_backward,
                               (m(Z), m(Z), w, 4, 64, FAKE, None, m(Z), m(Z), 0, FAKE, ws))):
            with pytest.raises(Z.ZeroError, match=f"{call}: weight") as e:
                f(*args, stream=0)
            assert e.value.code == Z.ZERO_EINVAL

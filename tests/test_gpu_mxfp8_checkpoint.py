"""8-bit activation checkpoints on the GPU: codes and exponents bit for bit as
the oracle's, decoded values exact, from any start and stride."""

import numpy as np
import pytest
import torch

import memory_reduced_muon_gb300 as q
from oracle import activations as act

from gpu_util import Guarded
from test_gpu_embedding import DT, Matrix, _np

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32, 0, 0), (5, 64, 0, 0), (3, 96, 8, 0), (7, 160, 16, 16), (33, 4096, 0, 0), (19, 2080, 1, 0), (257, 320, 3, 1), (2, 32, 0, 1)]


def _values(rows, cols, dtype, seed):
    """Values of all magnitudes, with blocks of zeros, of one value, at the borders of codes and of exponents."""
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x = x * torch.exp2(torch.randint(-10, 5, (rows, cols // 32, 1), generator=gen, device="cuda").float()).expand(-1, -1, 32).reshape(rows, cols)
    if rows > 2:
        x[0] = 0.0
        x[1] = torch.where(torch.arange(cols, device="cuda") % 2 == 0, 1.75, -1.8125)     # 448 2^-8 and a tie above it
        x[2, :32] = 2.0 ** -14
    return x.to(DT[dtype])


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pay_off", [0, 16])
def test_encode_and_decode(shape, dtype, pay_off):
    rows, cols, pad, off = shape
    x = Matrix(rows, cols, pad, DT[dtype], off, _values(rows, cols, dtype, 1))
    pay, sc = Guarded((rows * cols + pay_off,), torch.uint8), Guarded((rows, cols // 32), torch.uint8)
    q.qmuon_mxfp8_encode(x.t, pay.t[pay_off:], sc.t, rows, cols, dtype, ld_x=x.ld)
    back = Matrix(rows, cols, pad, DT[dtype], off)
    q.qmuon_mxfp8_decode(pay.t[pay_off:], sc.t, back.t, rows, cols, dtype, ld_x=back.ld)
    torch.cuda.synchronize()
    for m in (x, pay, sc, back):
        m.check()
    payload, scale = act.encode(x.t.float().cpu().numpy())
    got = pay.t[pay_off:].view(rows, cols).cpu().numpy()
    np.testing.assert_array_equal(sc.t.cpu().numpy(), scale)
    np.testing.assert_array_equal(got, payload)
    want = torch.from_numpy(act.decode64(payload, scale))
    np.testing.assert_array_equal(_np(back.t), want.to(DT[dtype]).double().numpy())
    if dtype != "f16":
        np.testing.assert_array_equal(_np(back.t), want.numpy())        # exact


@pytest.mark.parametrize("off", [0, 1])       # by vectors, and by elements
def test_all_codes_under_all_exponents(off):
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(256)
    scale = torch.arange(256, device="cuda", dtype=torch.uint8).repeat_interleave(8)
    want = act.decode64(codes.view(256, 256).cpu().numpy(), np.minimum(scale.view(256, 8).cpu().numpy(), 254))
    want[255] = np.nan                                                   # exponent byte 255 is no number
    for dtype in ("f32", "bf16", "f16"):
        x = Matrix(256, 256, 0, DT[dtype], off)
        q.qmuon_mxfp8_decode(codes, scale, x.t, 256, 256, dtype)
        torch.cuda.synchronize()
        x.check()
        got = x.t.double().cpu().numpy()
        with np.errstate(over="ignore"):
            f32 = want.astype(np.float32)                                # 448 2^127 is beyond fp32
            ref = torch.from_numpy(f32)
            if dtype == "f16":
                ref = torch.where(torch.isfinite(ref), ref.clamp(-65504, 65504), ref)
            np.testing.assert_array_equal(got, ref.to(DT[dtype]).double().numpy())


@pytest.mark.parametrize("off", [0, 1])
def test_values_that_are_not_finite(off):
    x = torch.ones(4, 32)
    x[0, 3] = float("nan")
    x[1] = float("nan")
    x[2, 5] = float("inf")
    x[3, 7] = -float("inf")
    m = Matrix(4, 32, 0, torch.float32, off, x.cuda())
    pay, sc = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, dtype=torch.uint8, device="cuda")
    q.qmuon_mxfp8_encode(m.t, pay, sc, 4, 32, "f32")
    back = torch.empty(4, 32, device="cuda")
    q.qmuon_mxfp8_decode(pay, sc, back, 4, 32, "f32")
    assert sc.flatten().tolist() == [119, 127, 254, 254]                 # 1 = 256 2^-8; nothing but NaN: as zeros; infinities
    assert bool(torch.isnan(back[0, 3])) and bool((back[0, :3] == 1).all()) and bool(torch.isnan(back[1]).all())
    assert float(back[2, 5]) == float("inf") and float(back[3, 7]) == -float("inf")


def test_the_norm_writes_the_same_checkpoint():
    rows, cols = 37, 256
    gen = torch.Generator("cuda").manual_seed(3)
    x, gain = torch.randn(rows, cols, generator=gen, device="cuda"), torch.rand(cols, generator=gen, device="cuda")
    y = torch.empty_like(x)
    pays = [torch.empty(rows, cols, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scs = [torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q.qmuon_rmsnorm_forward(x, gain, rows, cols, "f32", 1e-5, y=y, payload=pays[0], scale_inv=scs[0])
    q.qmuon_mxfp8_encode(y, pays[1], scs[1], rows, cols, "f32")          # y in fp32 is what the norm encodes
    assert torch.equal(*pays) and torch.equal(*scs)

"""GPU parity of the 8-bit block operators: quantise, restore, matrix product.

The references are written from the definitions in fp64 (tests/f8_ref.py).
Codes and scales have to be equal.  Products: the codes' products are exact in
fp32 (8 significant bits), so the error of an fp32 output is that of its sums;
with fp32 sums of k terms in any order it is at most about k 2^-24 of the sum of
the magnitudes, and for random signs sqrt(k) 2^-24; one more rounding for each
scale product and each block's sum.  The bound asserted is
(k + 4 kb) 2^-24 sum |a b| per element, and for bf16 outputs 2^-8 |c| on top.
"""

import numpy as np
import pytest
import torch

import f8_ref as R
from bit_nf4_quantized_17_b200 import qlora as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
LAYOUT = {"rows": Q.QLORA_F8_ROWS, "tiles": Q.QLORA_F8_TILES}
FORMAT = {"e4m3": Q.QLORA_E4M3, "e5m2": Q.QLORA_E5M2}


def _x(rows, cols, seed, dtype):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * np.exp2(g.integers(-12, 13, (rows, 1)))
    x[g.random((rows, cols)) < 0.01] *= 30
    x[g.random((rows, cols)) < 0.05] = 0
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("by", ["rows", "tiles"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 200), (130, 264), (257, 513),
                                       (33, 1030), (300, 1024)])
def test_quantize_and_restore(by, fmt, pow2, dtype, rows, cols):
    x = _x(rows, cols, rows * 1000 + cols, dtype)
    q = Q.qlora_f8_quantize(x.to(DEV), LAYOUT[by], FORMAT[fmt], pow2)
    codes, scales = R.quantize(x, by, fmt, pow2)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.values.float().cpu().numpy(), codes)
    pad = q.codes[:, cols:].cpu().numpy()
    assert not pad.any()
    want = R.restore(codes, scales, by)
    np.testing.assert_array_equal(Q.qlora_f8_dequantize(q, torch.float32).cpu().numpy(), want)
    np.testing.assert_array_equal(Q.qlora_f8_dequantize(q).float().cpu().numpy(),
                                  torch.from_numpy(want).bfloat16().float().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("by", ["rows", "tiles"])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_edges(fmt, by, pow2):
    """Zeros, the smallest and largest fp32 values, NaN and infinities, ties of the format."""
    x = torch.zeros(6, 384)
    x[1, :128] = torch.from_numpy(np.exp2(np.arange(128) - 149.0)).float()
    x[2, :128] = torch.finfo(torch.float32).max
    x[2, 5] = -torch.finfo(torch.float32).max
    x[3, 0], x[3, 1], x[3, 2], x[3, 3] = float("nan"), float("inf"), -float("inf"), 3.0
    x[3, 128] = float("inf")
    # midpoints of neighbouring codes, and the values just above and below
    f = R.FMAX[fmt]
    mids = torch.tensor(R.midpoints(fmt))[:120]
    x[4, :mids.numel()], x[4, 120] = mids, f
    x[5, :mids.numel()], x[5, 120] = torch.nextafter(mids, torch.tensor(0.0)), f
    if by == "tiles":
        x[2] = 0  # one scale for all rows
    q = Q.qlora_f8_quantize(x.to(DEV), LAYOUT[by], FORMAT[fmt], pow2)
    codes, scales = R.quantize(x, by, fmt, pow2)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.values.float().cpu().numpy(), codes)
    assert np.isnan(codes[3, :3]).all() and np.isfinite(codes[3, 3:128]).all()


def _matrices(m, n, k, trans, fa, fb, pow2, seed):
    a = Q.qlora_f8_quantize(_x(m, k, seed, torch.float32).to(DEV), Q.QLORA_F8_ROWS, FORMAT[fa],
                            pow2)
    b = _x(n, k, seed + 1, torch.float32) if trans else _x(k, n, seed + 1, torch.float32)
    return a, Q.qlora_f8_quantize(b.to(DEV), Q.QLORA_F8_TILES, FORMAT[fb], pow2)


def _dense(q, by):
    return R.restore(q.values.float().cpu().numpy(), q.scales.cpu().numpy(), by, np.float64)


def _check_product(a, b, trans, out):
    x, w = _dense(a, "rows"), _dense(b, "tiles")
    w = w.T if trans else w
    want, size = x @ w, np.abs(x) @ np.abs(w)
    k = x.shape[1]
    bound = (k + 4 * (k // 128 + 1)) * 2.0 ** -24 * size
    if out.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(want)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound + 1e-300).all(), float((np.abs(got - want) / (bound + 1e-300)).max())


SHAPES = [(1, 16, 16), (1, 128, 128), (1, 1000, 4096), (5, 4104, 1111), (16, 256, 1408),
          (17, 130, 129), (31, 640, 2048), (33, 384, 300), (64, 1000, 2560), (65, 128, 64),
          (128, 128, 1024), (130, 257, 700), (300, 1001, 1111), (512, 512, 8192),
          (1000, 136, 264),
          # more 128 x 128 tiles than SMs: CTA pairs, more than one tile a pair, ragged edges
          (2000, 2600, 640), (1500, 1701, 1111), (4300, 4104, 392), (6000, 1030, 100)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("trans", [True, False])
def test_matmul(m, n, k, trans):
    for fa, fb, pow2, dtype in (("e4m3", "e4m3", False, torch.float32),
                                ("e5m2", "e4m3", True, torch.bfloat16),
                                ("e4m3", "e5m2", False, torch.bfloat16)):
        a, b = _matrices(m, n, k, trans, fa, fb, pow2, m + n + k)
        guard = torch.full((m * n + 256,), 7.0, dtype=dtype, device=DEV)
        out = guard[128:128 + m * n].view(m, n)
        Q.qlora_f8_matmul(a, b, trans, out=out)
        _check_product(a, b, trans, out)
        assert (guard[:128] == 7).all() and (guard[128 + m * n:] == 7).all()

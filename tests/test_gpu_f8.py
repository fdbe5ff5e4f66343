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


@pytest.mark.parametrize("m,n,k", [(7, 300, 520), (70, 300, 520), (2500, 2304, 400)])
@pytest.mark.parametrize("trans", [True, False])
def test_bad_values_stay_in_their_row_and_column(m, n, k, trans):
    """NaN and infinities of A spoil their rows of C, those of B their columns, nothing else."""
    x = _x(m, k, 1, torch.float32)
    w = _x(n, k, 2, torch.float32)
    clean = Q.qlora_f8_matmul(
        Q.qlora_f8_quantize(x.to(DEV)),
        Q.qlora_f8_quantize((w if trans else w.t().contiguous()).to(DEV), Q.QLORA_F8_TILES), trans)
    x[3, 5], x[m - 1, k - 1] = float("nan"), float("inf")
    w[4, 130], w[n - 1, 0] = -float("inf"), float("nan")
    a = Q.qlora_f8_quantize(x.to(DEV))
    b = Q.qlora_f8_quantize((w if trans else w.t().contiguous()).to(DEV), Q.QLORA_F8_TILES)
    got = Q.qlora_f8_matmul(a, b, trans).float().cpu().numpy()
    bad = np.zeros((m, n), bool)
    bad[[3, m - 1]] = True
    bad[:, [4, n - 1]] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    # a spoilt value leaves the scale of its block to the others: the rest may move where it
    # was the block's largest, by a rounding of the codes (2^-4 of a value) at most
    rest = clean.float().cpu().numpy()
    scale = np.abs(R.restore(np.nan_to_num(a.values.float().cpu().numpy()), a.scales.cpu().numpy(),
                             "rows", np.float64)) @ np.abs(np.nan_to_num(w.numpy().T, posinf=0, neginf=0))
    assert (np.abs(got - rest)[~bad] <= 0.3 * scale[~bad] + 1e-30).all()


@pytest.mark.parametrize("m,n,k,trans", [(1, 1000, 300, True), (40, 500, 300, False),
                                         (2500, 2304, 400, True), (2500, 2304, 400, False)])
def test_padding_is_not_read(m, n, k, trans):
    """Rows of codes padded with NaN bytes, a larger ld than needed: the same product."""
    a, b = _matrices(m, n, k, trans, "e4m3", "e4m3", False, 5)
    want = Q.qlora_f8_matmul(a, b, trans)

    def padded(q):
        codes = torch.full((q.rows, q.codes.shape[1] + 32), 0x7f, dtype=torch.uint8, device=DEV)
        codes[:, :q.cols] = q.codes[:, :q.cols]
        return Q.F8Matrix(q.rows, q.cols, q.layout, q.format, q.pow2, codes, q.scales)
    assert torch.equal(Q.qlora_f8_matmul(padded(a), padded(b), trans), want)
    assert torch.equal(Q.qlora_f8_dequantize(padded(a)), Q.qlora_f8_dequantize(a))


def test_two_streams_at_once():
    """Calls without a workspace share nothing: two streams, interleaved, give what one gives."""
    sets = [_matrices(m, 1024, 2048, True, "e4m3", "e4m3", False, m) for m in (4, 100, 1500, 3000)]
    want = [Q.qlora_f8_matmul(a, b) for a, b in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(4):
        for j, (a, b) in enumerate(sets):
            s = streams[(i + j) % 2]
            got.append((j, Q.qlora_f8_matmul(a, b, stream=s), Q.qlora_f8_dequantize(a, stream=s)))
    torch.cuda.synchronize()
    for j, c, x in got:
        assert torch.equal(c, want[j])
        assert torch.equal(x, Q.qlora_f8_dequantize(sets[j][0]))


@pytest.mark.parametrize("m,n,k,trans", [(2500, 2568, 1111, True), (2500, 2568, 1111, False),
                                         (4300, 4105, 130, True), (2304, 4096, 2048, False)])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2")])
def test_power_of_two_scales_on_the_tensor_core(m, n, k, trans, fa, fb):
    """The same matrices told to be powers of two or not: the same sums, up to their order.
    Scales from 2^-126 (rows of zeros) to large ones, blocks past a group of four."""
    x, w = _x(m, k, 21, torch.float32), _x(n, k, 22, torch.float32)
    x[5] = 0
    x[6, :128] *= 2.0 ** 60
    x[7] *= 2.0 ** -100
    w = w if trans else w.t().contiguous()
    a = Q.qlora_f8_quantize(x.to(DEV), Q.QLORA_F8_ROWS, FORMAT[fa], True)
    b = Q.qlora_f8_quantize(w.to(DEV), Q.QLORA_F8_TILES, FORMAT[fb], True)
    told = Q.qlora_f8_matmul(a, b, trans, torch.float32)
    as_any = [Q.F8Matrix(q.rows, q.cols, q.layout, q.format, False, q.codes, q.scales)
              for q in (a, b)]
    untold = Q.qlora_f8_matmul(*as_any, trans, torch.float32)
    _check_product(a, b, trans, told)
    _check_product(a, b, trans, untold)
    assert (told[5] == 0).all() and (untold[5] == 0).all()
    mixed = Q.qlora_f8_matmul(a, as_any[1], trans, torch.float32)  # one of the two is told
    assert torch.equal(mixed, untold)


def test_deterministic_and_out():
    a, b = _matrices(33, 640, 4096, True, "e4m3", "e4m3", False, 3)
    c = Q.qlora_f8_matmul(a, b, dtype=torch.float32)
    out = torch.empty_like(c)
    assert Q.qlora_f8_matmul(a, b, out=out) is out and torch.equal(out, c)
    with pytest.raises(ValueError):
        Q.qlora_f8_matmul(a, b, out=torch.empty(640, 33, device=DEV))
    with pytest.raises(ValueError):
        Q.qlora_f8_matmul(a, b, out=torch.empty(33, 640, dtype=torch.float16, device=DEV))
    with pytest.raises(Q.QloraError):
        Q.qlora_f8_matmul(b, a.__class__.empty(33, 4096, Q.QLORA_F8_TILES))  # b is not by rows
    x = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError):
        Q.qlora_f8_quantize(x, out=Q.F8Matrix.empty(5, 64))
    with pytest.raises(ValueError):
        Q.qlora_f8_quantize(x[:, ::2])
    with pytest.raises(ValueError):
        Q.qlora_f8_quantize(x.half())


def test_past_32_bits():
    """More than 2^31 elements: quantise, restore and both products, checked on the last rows
    and columns against the same rows and columns alone."""
    m, n, k = 66000, 33008, 256
    g = torch.Generator(DEV).manual_seed(1)
    big = torch.randn(m, n, generator=g, device=DEV, dtype=torch.bfloat16)
    q = Q.qlora_f8_quantize(big, pow2=True)
    tail = Q.qlora_f8_quantize(big[-300:].contiguous(), pow2=True)
    assert torch.equal(q.codes[-300:], tail.codes)
    assert torch.equal(q.scales[:, -300:], tail.scales)
    assert torch.equal(Q.qlora_f8_dequantize(q)[-300:], Q.qlora_f8_dequantize(tail))
    t = Q.qlora_f8_quantize(big[:128 * 515], Q.QLORA_F8_TILES)
    tt = Q.qlora_f8_quantize(big[128 * 512:128 * 515].contiguous(), Q.QLORA_F8_TILES)
    assert torch.equal(t.codes[128 * 512:], tt.codes) and torch.equal(t.scales[512:], tt.scales)
    del big, t
    a = Q.qlora_f8_quantize(torch.randn(m, k, generator=g, device=DEV))
    b = Q.qlora_f8_quantize(torch.randn(n, k, generator=g, device=DEV), Q.QLORA_F8_TILES)
    c = Q.qlora_f8_matmul(a, b)  # 2.2e9 outputs

    def rows(x, at):
        return Q.F8Matrix(x.rows - at, x.cols, x.layout, x.format, x.pow2, x.codes[at:].contiguous(),
                          x.scales[:, at:].contiguous())
    assert torch.equal(c[65536:], Q.qlora_f8_matmul(rows(a, 65536), b))
    del c
    # a left operand of more than 2^31 codes against few columns, both directions' contraction
    w = Q.qlora_f8_quantize(torch.randn(64, n, generator=g, device=DEV), Q.QLORA_F8_TILES)
    y = Q.qlora_f8_matmul(q, w, dtype=torch.float32)
    want = Q.qlora_f8_matmul(rows(q, 65792), w, dtype=torch.float32)
    assert float((y[65792:] - want).abs().max()) <= 1e-5 * float(want.abs().max())

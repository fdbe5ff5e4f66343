"""Host-side checks of the 8-bit operators: sizes, refusals before any launch (no GPU needed),
and the reference's own rounding against torch's 8-bit types."""

import ctypes

import numpy as np
import pytest
import torch

import f8_ref as R
from bit_nf4_quantized_17_b200 import qlora as Q

BUF = 4096  # a fake, aligned device address: these calls return before they use it


def _m(rows=64, cols=256, layout=Q.QLORA_F8_ROWS, format=Q.QLORA_E4M3, ld=None, pow2=0,
       codes=BUF, scales=BUF):
    return Q.qlora_f8(rows, cols, cols if ld is None else ld, layout, format, pow2, 0, codes,
                      scales)


def test_sizes():
    assert Q.qlora_f8_sizes(5, 130, Q.QLORA_F8_ROWS) == {"ld": 144, "codes": 720, "scales": 40}
    assert Q.qlora_f8_sizes(129, 256, Q.QLORA_F8_TILES) == {"ld": 256, "codes": 33024,
                                                            "scales": 16}
    assert Q.qlora_f8_sizes(0, 1, Q.QLORA_F8_ROWS) == {"ld": 16, "codes": 0, "scales": 0}
    for rows, cols, layout, st in ((-1, 8, 0, Q.QLORA_ERR_SHAPE), (8, 0, 0, Q.QLORA_ERR_SHAPE),
                                   ((1 << 30) + 1, 1, 0, Q.QLORA_ERR_SHAPE),
                                   (1, (1 << 30) + 1, 0, Q.QLORA_ERR_SHAPE),
                                   (1 << 20, 1 << 20, 0, Q.QLORA_ERR_SHAPE),
                                   (8, 8, 2, Q.QLORA_ERR_UNSUPPORTED)):
        with pytest.raises(Q.QloraError) as e:
            Q.qlora_f8_sizes(rows, cols, layout)
        assert e.value.status == st


BAD = [
    (dict(cols=0), Q.QLORA_ERR_SHAPE), (dict(rows=-1), Q.QLORA_ERR_SHAPE),
    (dict(ld=255), Q.QLORA_ERR_SHAPE), (dict(ld=248), Q.QLORA_ERR_SHAPE),
    (dict(ld=264), Q.QLORA_ERR_SHAPE), (dict(layout=2), Q.QLORA_ERR_UNSUPPORTED),
    (dict(format=2), Q.QLORA_ERR_UNSUPPORTED), (dict(pow2=2), Q.QLORA_ERR_UNSUPPORTED),
    (dict(codes=None), Q.QLORA_ERR_NULL), (dict(scales=None), Q.QLORA_ERR_NULL),
    (dict(codes=BUF + 8), Q.QLORA_ERR_ALIGN), (dict(scales=BUF + 4), Q.QLORA_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD)
def test_matrix_refused_everywhere(kw, status):
    L, bad, good = Q.lib(), _m(**kw), _m()
    tiles = _m(layout=Q.QLORA_F8_TILES)
    assert L.qlora_f8_quantize(BUF, 0, bad, None) == status
    assert L.qlora_f8_dequantize(bad, BUF, 0, None) == status
    assert L.qlora_f8_matmul(bad, tiles, 1, BUF, 0, None) == status
    assert L.qlora_f8_matmul(good, _m(**{"layout": Q.QLORA_F8_TILES, **kw}), 1, BUF, 0,
                             None) == status


def test_call_refusals():
    L, a = Q.lib(), _m()
    b = _m(layout=Q.QLORA_F8_TILES)
    null = ctypes.POINTER(Q.qlora_f8)()
    assert L.qlora_f8_quantize(BUF, 0, null, None) == Q.QLORA_ERR_NULL
    assert L.qlora_f8_quantize(None, 0, a, None) == Q.QLORA_ERR_NULL
    assert L.qlora_f8_quantize(BUF + 2, 1, a, None) == Q.QLORA_ERR_ALIGN
    assert L.qlora_f8_quantize(BUF, 2, a, None) == Q.QLORA_ERR_UNSUPPORTED
    assert L.qlora_f8_dequantize(a, None, 0, None) == Q.QLORA_ERR_NULL
    assert L.qlora_f8_dequantize(a, BUF, 5, None) == Q.QLORA_ERR_UNSUPPORTED
    assert L.qlora_f8_dequantize(a, BUF + 4, 0, None) == Q.QLORA_ERR_ALIGN
    assert L.qlora_f8_matmul(null, b, 1, BUF, 0, None) == Q.QLORA_ERR_NULL
    assert L.qlora_f8_matmul(a, null, 1, BUF, 0, None) == Q.QLORA_ERR_NULL
    assert L.qlora_f8_matmul(a, b, 1, None, 0, None) == Q.QLORA_ERR_NULL
    assert L.qlora_f8_matmul(a, b, 1, BUF + 8, 0, None) == Q.QLORA_ERR_ALIGN
    assert L.qlora_f8_matmul(a, b, 1, BUF, 7, None) == Q.QLORA_ERR_UNSUPPORTED
    assert L.qlora_f8_matmul(a, a, 1, BUF, 0, None) == Q.QLORA_ERR_UNSUPPORTED
    assert L.qlora_f8_matmul(b, b, 1, BUF, 0, None) == Q.QLORA_ERR_UNSUPPORTED
    # contraction lengths: A is 64 x 256, B 64 x 256
    assert L.qlora_f8_matmul(a, b, 0, BUF, 0, None) == Q.QLORA_ERR_SHAPE
    assert L.qlora_f8_matmul(a, _m(cols=272, layout=Q.QLORA_F8_TILES), 1, BUF, 0,
                             None) == Q.QLORA_ERR_SHAPE
    assert L.qlora_f8_matmul(a, _m(rows=0, layout=Q.QLORA_F8_TILES), 1, BUF, 0,
                             None) == Q.QLORA_ERR_SHAPE
    # no rows: nothing to do, nothing asked of the pointers
    empty = _m(rows=0, codes=None, scales=None)
    assert L.qlora_f8_quantize(None, 0, empty, None) == Q.QLORA_OK
    assert L.qlora_f8_dequantize(empty, None, 0, None) == Q.QLORA_OK
    assert L.qlora_f8_matmul(empty, b, 1, None, 0, None) == Q.QLORA_OK


def _lin(L, bwd, W=None, A=BUF, B=BUF, r=16, x8=None, X=BUF, U=BUF, Y=BUF, dA=BUF, dB=BUF,
         grad=Q.QLORA_E5M2, ws=BUF, nbytes=1 << 30):
    W = W if W is not None else _m(256, 128, Q.QLORA_F8_TILES)
    x8 = x8 if x8 is not None else _m(32, 128)
    if bwd:
        return L.qlora_f8_linear_bwd(W, A, B, r, 1.0, x8, U, Y, grad, X, dA, dB, 0, ws, nbytes,
                                     None)
    return L.qlora_f8_linear_fwd(W, A, B, r, 1.0, X, x8, Y, U, ws, nbytes, None)


def test_linear_refusals():
    L = Q.lib()
    both = [
        (dict(A=None), Q.QLORA_ERR_NULL), (dict(B=None), Q.QLORA_ERR_NULL),
        (dict(ws=None), Q.QLORA_ERR_NULL), (dict(Y=None), Q.QLORA_ERR_NULL),
        (dict(A=BUF + 8), Q.QLORA_ERR_ALIGN), (dict(U=BUF + 4), Q.QLORA_ERR_ALIGN),
        (dict(ws=BUF + 8), Q.QLORA_ERR_ALIGN), (dict(X=BUF + 2), Q.QLORA_ERR_ALIGN),
        (dict(r=0), Q.QLORA_ERR_SHAPE), (dict(r=257), Q.QLORA_ERR_SHAPE),
        (dict(r=12), Q.QLORA_ERR_UNSUPPORTED),
        (dict(W=_m(252, 128, Q.QLORA_F8_TILES)), Q.QLORA_ERR_UNSUPPORTED),
        (dict(W=_m(256, 124, Q.QLORA_F8_TILES, ld=128), x8=_m(32, 124, ld=128)),
         Q.QLORA_ERR_UNSUPPORTED),
        (dict(W=_m(256, 128)), Q.QLORA_ERR_UNSUPPORTED),
        (dict(x8=_m(32, 128, Q.QLORA_F8_TILES)), Q.QLORA_ERR_UNSUPPORTED),
        (dict(x8=_m(32, 256)), Q.QLORA_ERR_SHAPE),
        (dict(W=_m(0, 128, Q.QLORA_F8_TILES)), Q.QLORA_ERR_SHAPE),
        (dict(nbytes=256), Q.QLORA_ERR_WORKSPACE),
    ]
    for bwd in (False, True):
        for kw, status in both:
            assert _lin(L, bwd, **kw) == status, (bwd, kw)
    assert _lin(L, False, X=None) == Q.QLORA_ERR_NULL
    for kw, status in ((dict(U=None), Q.QLORA_ERR_NULL), (dict(dA=None), Q.QLORA_ERR_NULL),
                       (dict(dB=None), Q.QLORA_ERR_NULL), (dict(dA=BUF + 8), Q.QLORA_ERR_ALIGN),
                       (dict(grad=2), Q.QLORA_ERR_UNSUPPORTED)):
        assert _lin(L, True, **kw) == status, kw
    assert _lin(L, False, x8=_m(0, 128, codes=None, scales=None)) == Q.QLORA_OK


def test_kept_input_refusals():
    L = Q.lib()

    def call(q=None, x8=None, r=16, U=BUF, dY=BUF, dA=BUF, dB=BUF, ws=BUF, nbytes=1 << 30, opts=None):
        q = q or Q.qlora_nf4(256, 128, 64, 256, 0, 0, BUF, BUF, BUF, BUF)
        return L.qlora_linear_bwd_f8(q, BUF, BUF, r, 1.0, opts, x8 or _m(32, 128), U, dY, BUF, dA,
                                     dB, 0, ws, nbytes, None)
    for kw, status in ((dict(U=None), Q.QLORA_ERR_NULL), (dict(dY=None), Q.QLORA_ERR_NULL),
                       (dict(dA=None), Q.QLORA_ERR_NULL), (dict(ws=None), Q.QLORA_ERR_NULL),
                       (dict(dB=BUF + 8), Q.QLORA_ERR_ALIGN), (dict(r=0), Q.QLORA_ERR_SHAPE),
                       (dict(x8=_m(32, 256)), Q.QLORA_ERR_SHAPE),
                       (dict(x8=_m(32, 128, Q.QLORA_F8_TILES)), Q.QLORA_ERR_UNSUPPORTED),
                       (dict(x8=_m(32, 128, codes=None)), Q.QLORA_ERR_NULL),
                       (dict(nbytes=Q.qlora_linear_bwd_f8_workspace(32, 256, 128, 16) - 1),
                        Q.QLORA_ERR_WORKSPACE),
                       (dict(opts=Q.qlora_adapter_opts(2, 0, None, 0.0, 0, None, None)),
                        Q.QLORA_ERR_NULL),
                       (dict(opts=Q.qlora_adapter_opts(1, 0, None, 1.0, 0, BUF, None)),
                        Q.QLORA_ERR_UNSUPPORTED)):
        assert call(**kw) == status, kw


def test_workspace_queries():
    for M in (0, 1, 16, 17, 5000):
        f, b = Q.qlora_f8_linear_workspace(M, 256, 128, 16)
        assert 256 <= f <= b
        assert Q.qlora_linear_bwd_f8_workspace(M, 256, 128, 16) >= \
            Q.qlora_linear_workspace(M, 256, 128, 16)[1]
        # a rank that the CUDA-core path takes: X restored in bf16
        assert Q.qlora_linear_bwd_f8_workspace(M, 256, 128, 5) >= \
            Q.qlora_linear_workspace(M, 256, 128, 5)[1] + 2 * M * 128
    for args in ((-1, 8, 8, 8), (1, 0, 8, 8), (1, 8, 8, 257), ((1 << 30) + 1, 8, 8, 8)):
        with pytest.raises(Q.QloraError) as e:
            Q.qlora_f8_linear_workspace(*args)
        assert e.value.status == Q.QLORA_ERR_SHAPE


def test_binding_refusals():
    u8 = torch.uint8
    good = dict(rows=4, cols=130, layout=Q.QLORA_F8_ROWS, format=Q.QLORA_E4M3, pow2=False,
                codes=torch.zeros(4, 144, dtype=u8), scales=torch.zeros(2, 4))
    q = Q.F8Matrix(**good)
    assert q.values.shape == (4, 130) and q.nbytes == 4 * 144 + 32
    for kw in (dict(codes=torch.zeros(4, 136, dtype=u8)), dict(codes=torch.zeros(4, 128, dtype=u8)),
               dict(codes=torch.zeros(4, 144)), dict(scales=torch.zeros(4, 2)),
               dict(scales=torch.zeros(2, 4, dtype=torch.float64)), dict(layout=5), dict(format=9),
               dict(codes=torch.zeros(4, 288, dtype=u8)[:, ::2])):
        with pytest.raises(ValueError):
            Q.F8Matrix(**{**good, **kw})
    with pytest.raises(ValueError):
        Q.qlora_f8_quantize(torch.zeros(4, 4))  # not on a GPU
    w = Q.F8Matrix.empty(8, 100, Q.QLORA_F8_TILES, device="cpu")
    with pytest.raises(ValueError):
        Q.qlora_f8_matmul(q, w)  # 130 against 100


@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_reference_rounding(fmt, dtype):
    """round8 against torch's conversion: every code, every midpoint, the values beside it."""
    mids = torch.from_numpy(R.midpoints(fmt).copy())
    x = torch.cat([mids, torch.nextafter(mids, torch.tensor(0.0)),
                   torch.nextafter(mids, torch.tensor(1e9)), torch.zeros(1),
                   torch.full((1,), R.FMAX[fmt])])
    x = torch.cat([x, -x])
    np.testing.assert_array_equal(R.round8(x.numpy(), fmt), x.to(dtype).double().numpy())

"""GPU: how close the fp32 outputs of the 8-bit layers are to fp64 as a whole, in the norm,
beside the bounds per element of test_gpu_f8_linear.py, which worst cases make wide.

What the bounds are made of, relative, for operands of random signs (B = 2^e m, m in [1, 2)):
  - dA reads V, and dB U, as three bf16 terms, 24 bits: as good as fp32.  (Of two, the second
    lies within 2^-8 2^e, evenly, 2^-8 / sqrt(3) in the mean square; its rounding is within 2^-8
    of its power of two, 0.72 2^-8 / sqrt(3) of itself. Together 3.7e-6 2^e, or 2.5e-6 of
    values whose mean square is 1.44 2^e.)
  - sums in TMEM are cut off: a chain of n additions loses about n 2^-24 2 / 3 of its sum
    (half a unit each of partial sums that grow with the square root), 2.5e-6 for the
    longest, 64, and 0.64e-6 for 16.
  - fp32 sums of the chains, a few 2^-24.
U and dB have the sums only: 2.5e-6 and a few 2^-24, within 3e-6 over any length.  dA has
V's and its own: in the mean square 3.6e-6, within 4e-6.  Where the chains end at 16 (few tokens,
for dA also few columns of dY) within 1.2e-6, which two terms do not reach.
"""

import pytest
import torch

from bit_nf4_quantized_17_b200 import qlora as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(M, N, K, r):
    g = torch.Generator(DEV).manual_seed(M + N + K + r)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return [t.bfloat16() for t in (rn(N, K) / 50, rn(r, K) / r ** 0.5, rn(N, r) / 50, rn(M, K),
                                   rn(M, N))]


def _product(a, b):
    """a^T b in fp64, a stretch of rows at a time."""
    out = torch.zeros(a.shape[1], b.shape[1], dtype=torch.float64, device=DEV)
    for i in range(0, a.shape[0], 4096):
        out += a[i:i + 4096].double().t() @ b[i:i + 4096].double()
    return out


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


WIDE = [(300, 22016, 16), (2048, 8192, 64), (16384, 22016, 64), (16384, 11008, 256),
        (10001, 5000, 136)]


@pytest.mark.parametrize("M,K,r", WIDE)
def test_factor_over_many_columns(M, K, r):
    W, A, B, X, _ = _inputs(M, 64, K, r)
    w8, U = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES), torch.empty((M, r), device=DEV)
    Q.qlora_f8_linear_fwd(w8, A, B, float(r), X, Q.F8Matrix.empty(M, K), U_save=U, check=True)
    assert _off(U, X.double() @ A.double().t()) < 3e-6


SHORT = [(2048, 256, 4096, 16), (1000, 64, 1024, 64), (1024, 200, 1024, 128),
         (300, 256, 2048, 24), (17, 256, 704, 256)]


@pytest.mark.parametrize("M,N,K,r", SHORT)
def test_grad_a_reads_all_of_v(M, N, K, r):
    W, A, B, X, dY = _inputs(M, N, K, r)
    w8, x8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES), Q.qlora_f8_quantize(X)
    want = _product(dY.double() @ B.double(), Q.qlora_f8_dequantize(x8))
    U = torch.zeros((M, r), device=DEV)
    _, dA, _ = Q.qlora_f8_linear_bwd(w8, A, B, float(r), x8, U, dY, check=True)
    assert _off(dA, want) < 1.2e-6
    q = Q.qlora_quantize(W)
    _, dA, _ = Q.qlora_linear_bwd_f8(q, A, B, r, float(r), x8, U, dY, check=True)
    assert _off(dA, want) < 1.2e-6


LONG = [(16384, 256, 4096, 16), (16384, 22016, 256, 64), (8192, 128, 11008, 32),
        (20001, 72, 2048, 128),
        (65536, 136, 1032, 64), (9000, 64, 11008, 256), (33000, 64, 200, 160)]


@pytest.mark.parametrize("M,N,K,r", LONG)
def test_grad_a_over_many_tokens(M, N, K, r):
    W, A, B, X, dY = _inputs(M, N, K, r)
    w8, x8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES), Q.qlora_f8_quantize(X)
    U = torch.zeros((M, r), device=DEV)
    _, dA, _ = Q.qlora_f8_linear_bwd(w8, A, B, float(r), x8, U, dY, want_dx=False, check=True)
    want = _product(dY.double() @ B.double(), Q.qlora_f8_dequantize(x8))
    assert _off(dA, want) < 4e-6
    # added to what is there, once
    dA2 = dA.clone()
    Q.qlora_f8_linear_bwd(w8, A, B, float(r), x8, U, dY, dA=dA2, accumulate=True, want_dx=False,
                          dB=torch.zeros((N, r), device=DEV), check=True)
    assert _off(dA2, 2 * want) < 4e-6
    if K % 64 == 0:
        # V is the NF4 layer's here, summed over d_out in one accumulator: N / 16 additions
        q = Q.qlora_quantize(W)
        _, dA, _ = Q.qlora_linear_bwd_f8(q, A, B, r, float(r), x8, U, dY, want_dx=False, check=True)
        assert _off(dA, want) < 4e-6 + N / 16 * 2.0 ** -24 * 2 / 3


@pytest.mark.parametrize("M,N,K,r", [(16384, 4096, 64, 16), (65536, 1000, 64, 64),
                                     (40001, 2048, 64, 96), (20000, 11008, 64, 128),
                                     (9000, 22016, 64, 64), (70000, 136, 64, 200),
                                     (33001, 4096, 64, 256)])
def test_grad_b_over_many_tokens(M, N, K, r):
    W, A, B, X, dY = _inputs(M, N, K, r)
    w8, x8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES), Q.qlora_f8_quantize(X)
    U = X.float() @ A.float().t()
    _, _, dB = Q.qlora_f8_linear_bwd(w8, A, B, float(r), x8, U, dY, want_dx=False, check=True)
    want = _product(dY, U)
    assert _off(dB, want) < 3e-6
    dB2 = dB.clone()
    Q.qlora_f8_linear_bwd(w8, A, B, float(r), x8, U, dY, dB=dB2, accumulate=True, want_dx=False,
                          dA=torch.zeros((r, K), device=DEV), check=True)
    assert _off(dB2, 2 * want) < 3e-6


@pytest.mark.parametrize("M,N,K,r", [(2048, 4096, 64, 16), (1000, 1032, 64, 64),
                                     (512, 200, 64, 128),
                                     (500, 256, 64, 24), (17, 264, 64, 256), (130, 8, 64, 72)])
def test_grad_b_reads_all_of_u(M, N, K, r):
    W, A, B, X, dY = _inputs(M, N, K, r)
    w8, x8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES), Q.qlora_f8_quantize(X)
    U = X.float() @ A.float().t()
    _, _, dB = Q.qlora_f8_linear_bwd(w8, A, B, float(r), x8, U, dY, check=True)
    assert _off(dB, _product(dY, U)) < 1.2e-6

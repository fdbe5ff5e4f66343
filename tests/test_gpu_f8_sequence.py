"""GPU: 8-bit calls one after another, nothing waiting between them, each launch overlapping the
tail of the one before: every call reads what the calls ahead of it wrote, none older."""

import pytest
import torch

from bit_nf4_quantized_17_b200 import qlora as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(DEV).manual_seed(seed), device=DEV)


@pytest.mark.parametrize("m,n,k,trans", [(12, 640, 2048, True), (200, 1024, 1024, True),
                                         (2304, 4096, 640, True), (2304, 4096, 640, False)])
@pytest.mark.parametrize("pow2", [False, True])
def test_scales_written_just_before(m, n, k, trans, pow2):
    """Both operands quantised anew, into the same arrays, right before each product: values
    whose scales differ from call to call."""
    a = Q.F8Matrix.empty(m, k, pow2=pow2)
    b = Q.F8Matrix.empty(*((n, k) if trans else (k, n)), Q.QLORA_F8_TILES, pow2=pow2)
    xs = [_randn(i, m, k) * 8.0 ** (i - 1) for i in range(3)]
    ws = [_randn(9 + i, b.rows, b.cols) * 4.0 ** (1 - i) for i in range(3)]

    def step(i, wait):
        Q.qlora_f8_quantize(ws[i], out=b)
        Q.qlora_f8_quantize(xs[i], out=a)
        if wait:
            torch.cuda.synchronize()
        return Q.qlora_f8_matmul(a, b, trans, torch.float32)
    want = [step(i, True) for i in range(3)]
    torch.cuda.synchronize()
    got = [(i % 3, step(i % 3, False)) for i in range(12)]
    for i, c in got:
        assert torch.equal(c, want[i])


def test_more_row_tiles_than_a_grid_has_rows():
    """More than 65535 tiles of 128 tokens: the last rows are those of the same tokens alone."""
    M, N, K, r, tail = 65535 * 128 + 333, 8, 16, 8, 300
    bf16 = torch.bfloat16
    A, B = (_randn(1, r, K) / 3).to(bf16), _randn(2, N, r).to(bf16)
    X, dY = _randn(3, M, K).to(bf16), _randn(4, M, N).to(bf16)
    w8 = Q.qlora_f8_quantize(_randn(5, N, K), Q.QLORA_F8_TILES)

    def run(x, dy):
        m = x.shape[0]
        x8, U = Q.F8Matrix.empty(m, K), torch.empty((m, r), device=DEV)
        Y = Q.qlora_f8_linear_fwd(w8, A, B, 16.0, x, x8, U_save=U, check=True)
        dX, _, _ = Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dy, check=True)
        return Y, U, x8.codes, x8.scales.t(), dX
    for got, alone in zip(run(X, dY), run(X[-tail:].contiguous(), dY[-tail:].contiguous())):
        assert torch.equal(got[-tail:], alone)

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

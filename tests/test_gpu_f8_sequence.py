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


def _layer(M, N, K, r, seed):
    """Operands of a layer over an 8-bit base, and a step with its own workspaces."""
    bf16 = torch.bfloat16
    A, B = (_randn(seed, r, K) / r ** 0.5).to(bf16), (_randn(seed + 1, N, r) / 50).to(bf16)
    X, dY = _randn(seed + 2, M, K).to(bf16), _randn(seed + 3, M, N).to(bf16)
    w8 = Q.qlora_f8_quantize(_randn(seed + 4, N, K) / 50, Q.QLORA_F8_TILES)
    x8, U = Q.F8Matrix.empty(M, K), torch.empty((M, r), device=DEV)

    def workspaces(fill):
        ws = [torch.full((max(n, 256),), fill, dtype=torch.uint8, device=DEV)
              for n in Q.qlora_f8_linear_workspace(M, N, K, r)]
        for w in ws:
            w[:256] = 0
        return ws

    def step(ws, stream=None):
        Y = Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U, workspace=ws[0], stream=stream)
        return [Y, *Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY, workspace=ws[1],
                                          stream=stream)]
    return step, workspaces(0), workspaces


def test_layers_on_two_streams_at_once():
    """Layers of every path, decoding and training, side by side on two streams: what each gives
    alone."""
    sets = [_layer(*s, 100 * i) for i, s in enumerate(
        [(9, 1024, 2048, 16), (2000, 512, 1024, 128), (300, 1000, 2048, 256), (24, 2048, 1024, 64),
         (1000, 2048, 640, 72), (200, 640, 4096, 32)])]
    want = [step(ws) for step, ws, _ in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        # a layer's calls share its outputs X8 and U: they stay on one stream
        got = [step(ws, streams[i % 2]) for i, (step, ws, _) in enumerate(sets)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


# one launch takes 8 splits x 64 tokens x 12 tiles and accumulator (rank 64: two in 256 TMEM
# columns, 12288 tokens) or 16 (rank 200: chunks of 112 ranks, two in 512 columns, 16384)
@pytest.mark.parametrize("M,N,K,r", [(13000, 136, 200, 64), (17000, 72, 136, 200)])
def test_gradients_of_several_launches_captured(M, N, K, r):
    """So many tokens that dA and dB are several launches that add: captured, replayed twice, with
    workspaces that hold anything, as eager calls with clean ones."""
    step, ws, workspaces = _layer(M, N, K, r, 7)
    want = [t.clone() for t in step(ws)]
    dirty = workspaces(0xff)
    n0 = Q.qlora_launch_count()
    step(dirty)
    assert Q.qlora_launch_count() - n0 > 7  # a step of one launch each
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(dirty)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)

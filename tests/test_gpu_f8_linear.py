"""GPU parity of the layers that use 8-bit matrices: the NF4 backward from an input kept in 8
bits, and the linear layer over an 8-bit base, against fp64 from the definitions (f8_ref.py).

Bounds, per element and derived before the first run (e = 2^-24, half an ulp of fp32; sums of
n terms in fp32 are off by at most n e times the sum of magnitudes):
  U   K e |x||A|^T
  dB  s (M e + 2^-16) |dY|^T |U|            U as bf16 hi + lo: 2^-17 relative
  dA  s (M e + N e + 2^-16) (|dY||B|)^T |X^|  V likewise
  Y   2^-8 |Y| + (K + 4 K/128 + 4) e |X^||W^|^T + s (K e + 2 r e + 2^-16) |x||A|^T |B|^T
  dX  the same with N for K
"""

import numpy as np
import pytest
import torch

import f8_ref as R
import oracle
from bit_nf4_quantized_17_b200 import qlora as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = 2.0 ** -24


def _rand(shape, seed, std=1.0, dtype=torch.bfloat16):
    g = np.random.default_rng(seed)
    x = g.standard_normal(shape) * std
    x[g.random(shape) < 0.01] *= 8
    return torch.from_numpy(x).to(dtype)


def _f(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _within(got, want, bound, name):
    got = _f(got)
    assert got.shape == want.shape and np.isfinite(got).all(), name
    worst = float((np.abs(got - want) / (bound + 1e-300)).max()) if got.size else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} of the bound"


def _rand_case(M, N, K, r, seed):
    return (_rand((N, K), seed, 0.02), _rand((r, K), seed + 1, r ** -0.5),
            _rand((N, r), seed + 2, 0.05), _rand((M, K), seed + 3), _rand((M, N), seed + 4))


def _grad_bounds(s, dy, b, u, xr):
    M, N = dy.shape
    v = dy @ b
    db = s * dy.T @ u
    da = s * v.T @ xr
    return (da, s * (M * E + N * E + 2.0 ** -16) * (np.abs(dy) @ np.abs(b)).T @ np.abs(xr),
            db, s * (M * E + 2.0 ** -16) * np.abs(dy).T @ np.abs(u))


CKPT = [(1, 64, 64, 8), (3, 80, 192, 5), (2, 512, 1024, 16), (16, 520, 2048, 136),
        (17, 200, 128, 16), (130, 96, 320, 64), (300, 1000, 640, 24), (600, 512, 1088, 256),
        (1000, 384, 704, 128)]


@pytest.mark.parametrize("M,N,K,r", CKPT)
@pytest.mark.parametrize("fmt,pow2", [(Q.QLORA_E4M3, False), (Q.QLORA_E4M3, True),
                                      (Q.QLORA_E5M2, False)])
def test_nf4_backward_from_kept_input(M, N, K, r, fmt, pow2):
    W, A, B, X, dY = _rand_case(M, N, K, r, M + N + K)
    q = Q.qlora_quantize(W.to(DEV))
    Ad, Bd, Xd, dYd = (t.to(DEV) for t in (A, B, X, dY))
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    Q.qlora_linear_fwd(q, Ad, Bd, 16.0, Xd, U_save=U)
    x8 = Q.qlora_f8_quantize(Xd, Q.QLORA_F8_ROWS, fmt, pow2)
    xr = _f(Q.qlora_f8_dequantize(x8))
    dX, dA, dB = Q.qlora_linear_bwd_f8(q, Ad, Bd, r, 16.0, x8, U, dYd, check=True)
    ref = Q.qlora_linear_bwd(q, Ad, Bd, 16.0, Xd, U, dYd, check=True)
    assert torch.equal(dX, ref[0]) and torch.equal(dB, ref[2])  # neither reads X
    da, ba, db, bb = _grad_bounds(16.0 / r, _f(dY), _f(B), _f(U), xr)
    _within(dA, da, ba, "dA")
    _within(dB, db, bb, "dB")
    # accumulated, and without dX
    A2, B2 = dA.clone(), dB.clone()
    none, _, _ = Q.qlora_linear_bwd_f8(q, Ad, Bd, r, 16.0, x8, U, dYd, dA=A2, dB=B2,
                                       accumulate=True, want_dx=False, check=True)
    assert none is None
    _within(A2, 2 * da, 2 * ba + 2 * E * np.abs(da), "dA + dA")
    _within(B2, 2 * db, 2 * bb + 2 * E * np.abs(db), "dB + dB")


@pytest.mark.parametrize("M", [13, 300])
def test_kept_input_with_adapters_and_dropout(M):
    """The kept form of x_drop, per-token adapters: as the bf16 call on the restored x_drop."""
    N, K, r, n, p = 512, 1024, 16, 3, 0.1
    W, A, B, X, dY = _rand_case(M, N, K, n * r, 9)
    q = Q.qlora_quantize(W.to(DEV))
    A, B, X, dY = (t.to(DEV) for t in (A, B, X, dY))
    ids = torch.from_numpy(np.random.default_rng(3).integers(-1, n, M).astype(np.int32)).to(DEV)
    mask = Q.dropout_keep_mask(M, K, p, torch.Generator(DEV).manual_seed(1))
    xd = torch.empty_like(X)
    U = torch.empty((M, n * r), dtype=torch.float32, device=DEV)
    Q.qlora_linear_fwd_ex(q, A, B, r, 16.0, X, adapter=ids, p=p, keep_mask=mask, x_drop=xd,
                          U_save=U, check=True)
    x8 = Q.qlora_f8_quantize(xd, pow2=True)
    got = Q.qlora_linear_bwd_f8(q, A, B, r, 16.0, x8, U, dY, adapter=ids, p=p, keep_mask=mask,
                                check=True)
    xr = Q.qlora_f8_dequantize(x8)
    ref = Q.qlora_linear_bwd_ex(q, A, B, r, 16.0, X, U, dY, adapter=ids, p=p, keep_mask=mask,
                                x_drop=xr, check=True)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])
    v = _f(dY) @ _f(B)
    for a in range(n):
        v[(ids.cpu().numpy() != a), a * r:(a + 1) * r] = 0
    s = 16.0 / r / (1 - p)
    bound = s * (M * E + N * E + 2.0 ** -16) * (np.abs(_f(dY)) @ np.abs(_f(B))).T @ np.abs(_f(xr))
    _within(got[1], s * v.T @ _f(xr), bound, "dA")


LIN = [(1, 64, 64, 8), (2, 200, 328, 16), (7, 4096, 1032, 16), (16, 256, 1408, 64),
       (17, 136, 128, 24), (40, 648, 2048, 64), (64, 1000, 264, 8), (65, 128, 64, 16),
       (130, 256, 704, 40), (300, 1000, 1112, 64), (700, 512, 1024, 136), (520, 1032, 904, 256),
       (1900, 1608, 1704, 72), (2100, 1504, 1800, 256)]


@pytest.mark.parametrize("M,N,K,r", LIN)
@pytest.mark.parametrize("grad,pow2", [(Q.QLORA_E5M2, False), (Q.QLORA_E4M3, True)])
def test_linear_over_8_bit_base(M, N, K, r, grad, pow2):
    W, A, B, X, dY = _rand_case(M, N, K, r, M + N + K + r)
    s = 16.0 / r
    w8 = Q.qlora_f8_quantize(W.to(DEV), Q.QLORA_F8_TILES, Q.QLORA_E4M3, pow2)
    Ad, Bd, Xd, dYd = (t.to(DEV) for t in (A, B, X, dY))
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    x8 = Q.F8Matrix.empty(M, K, pow2=pow2)
    Y = Q.qlora_f8_linear_fwd(w8, Ad, Bd, 16.0, Xd, x8, U_save=U, check=True)
    dX, dA, dB = Q.qlora_f8_linear_bwd(w8, Ad, Bd, 16.0, x8, U, dYd, grad, check=True)

    codes, scales = R.quantize(X, "rows", "e4m3", pow2)
    assert np.array_equal(_f(x8.values), codes) and np.array_equal(x8.scales.cpu().numpy(), scales)
    xq = R.restore(codes, scales, "rows", np.float64)
    wq = R.restore(*R.quantize(W, "tiles", "e4m3", pow2), "tiles", np.float64)
    dq = R.restore(*R.quantize(dY, "rows", "e5m2" if grad == Q.QLORA_E5M2 else "e4m3", pow2),
                   "rows", np.float64)
    a, b, x, dy = _f(A), _f(B), _f(X), _f(dY)
    u, size_u = x @ a.T, np.abs(x) @ np.abs(a).T
    _within(U, u, K * E * size_u, "U")
    y = xq @ wq.T + s * u @ b.T
    _within(Y, y, 2.0 ** -8 * np.abs(y) + (K + K // 32 + 4) * E * np.abs(xq) @ np.abs(wq).T
            + s * (K * E + 2 * r * E + 2.0 ** -16) * size_u @ np.abs(b).T, "Y")
    v, size_v = dy @ b, np.abs(dy) @ np.abs(b)
    dx = dq @ wq + s * v @ a
    _within(dX, dx, 2.0 ** -8 * np.abs(dx) + (N + N // 32 + 4) * E * np.abs(dq) @ np.abs(wq)
            + s * (N * E + 2 * r * E + 2.0 ** -16) * size_v @ np.abs(a), "dX")
    xr = torch.from_numpy(R.restore(codes, scales, "rows")).bfloat16().double().numpy()
    da, ba, db, bb = _grad_bounds(s, dy, b, _f(U), xr)
    _within(dA, da, ba, "dA")
    _within(dB, db, bb, "dB")


def test_no_tokens():
    W, A, B, X, dY = _rand_case(1, 64, 64, 8, 1)
    A, B = A.to(DEV), B.to(DEV)
    q = Q.qlora_quantize(W.to(DEV))
    w8 = Q.qlora_f8_quantize(W.to(DEV), Q.QLORA_F8_TILES)
    x8 = Q.F8Matrix.empty(0, 64)
    none = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    U = torch.empty((0, 8), dtype=torch.float32, device=DEV)
    assert Q.qlora_f8_linear_fwd(w8, A, B, 16.0, none, x8, U_save=U).shape == (0, 64)
    assert Q.qlora_f8_matmul(x8, w8).shape == (0, 64)
    for call in (lambda **k: Q.qlora_linear_bwd_f8(q, A, B, 8, 16.0, x8, U, none, **k),
                 lambda **k: Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, none, **k)):
        dA, dB = torch.ones((8, 64), device=DEV), torch.ones((64, 8), device=DEV)
        call(dA=dA, dB=dB, accumulate=True)
        assert (dA == 1).all() and (dB == 1).all()
        call(dA=dA, dB=dB)
        assert (dA == 0).all() and (dB == 0).all()


def _rel(got, want):
    return float(np.linalg.norm(_f(got) - want) / np.linalg.norm(want))


def test_run_together():
    """As they are used: train an adapter over NF4 with its inputs kept in 8 bits, merge it, put
    the merged weight into 8 bits, serve it, and train a second adapter over that base."""
    M, N, K, r = 200, 256, 384, 16
    W, A, B, X, dY = _rand_case(M, N, K, r, 5)
    A, B, X, dY = (t.to(DEV) for t in (A, B, X, dY))
    q = Q.qlora_quantize(W.to(DEV))
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    Q.qlora_linear_fwd(q, A, B, 16.0, X, U_save=U)
    x8 = Q.qlora_f8_quantize(X)
    _, dA, dB = Q.qlora_linear_bwd_f8(q, A, B, r, 16.0, x8, U, dY, check=True)
    exact = Q.qlora_linear_bwd(q, A, B, 16.0, X, U, dY, check=True)
    # a kept value is off by at most 2^-4 of itself: so is dA's sum of magnitudes
    v = np.abs(_f(dY) @ _f(B))
    bound = (2.0 ** -4 + 2.0 ** -8) * v.T @ np.abs(_f(X)) + 2.0 ** -4 * np.abs(_f(X)).max() * 0.01
    assert (np.abs(_f(dA) - _f(exact[1])) <= bound).all()
    assert torch.equal(dB, exact[2])
    merged = Q.qlora_merge(q, A, B, 16.0)
    w8 = Q.qlora_f8_quantize(merged, Q.QLORA_F8_TILES)
    y = Q.qlora_f8_matmul(x8, w8)
    # two operands with relative errors of at most 2^-4, independent of each other
    assert _rel(y, _f(X) @ _f(merged).T) < 0.06
    B0 = torch.zeros_like(B)
    y2 = Q.qlora_f8_linear_fwd(w8, A, B0, 16.0, X, Q.F8Matrix.empty(M, K), check=True)
    assert torch.equal(y2, y)  # an adapter whose B is zero adds nothing


def test_captured_and_replayed():
    """Forward and backward captured once, replayed on new inputs, beside an eager call."""
    M, N, K, r = 100, 256, 512, 16
    W, A, B, X, dY = (t.to(DEV) for t in _rand_case(M, N, K, r, 6))
    w8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES)
    q = Q.qlora_quantize(W)
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    x8 = Q.F8Matrix.empty(M, K)
    wf, wb = Q.qlora_f8_linear_workspace(M, N, K, r)
    wn = Q.qlora_linear_bwd_f8_workspace(M, N, K, r)
    ws = [torch.zeros(max(n, 256), dtype=torch.uint8, device=DEV) for n in (wf, wb, wn)]

    def step():
        Y = Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U, workspace=ws[0])
        g = Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY, workspace=ws[1])
        h = Q.qlora_linear_bwd_f8(q, A, B, r, 16.0, x8, U, dY, workspace=ws[2])
        return [Y, *g, *h]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    X.copy_(_rand((M, K), 77).to(DEV))
    dY.copy_(_rand((M, N), 78).to(DEV))
    graph.replay()
    first = [o.clone() for o in outs]
    graph.replay()
    eager = step()
    torch.cuda.synchronize()
    for a, b, c in zip(first, outs, eager):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_on_another_stream():
    """stream=: results equal, allocations in that stream's order, while the default stream is
    busy with other work."""
    M, N, K, r = 300, 512, 1024, 16
    W, A, B, X, dY = (t.to(DEV) for t in _rand_case(M, N, K, r, 8))
    w8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES)
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    s = torch.cuda.Stream()

    def step(stream):
        x8 = Q.F8Matrix.empty(M, K)
        Y = Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U, stream=stream)
        g = Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY, stream=stream)
        z = Q.qlora_f8_matmul(Q.qlora_f8_quantize(X, stream=stream), w8, stream=stream)
        return [Y, *g, z, Q.qlora_f8_dequantize(x8, stream=stream)]

    want = step(None)
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device=DEV)
    for _ in range(4):
        busy = busy @ busy
        busy /= busy.abs().max()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_gradients_against_differences():
    """dX, dA, dB of the layer over the 8-bit base against central differences of its loss in
    fp64, from the operands as they are held in 8 bits (the layer's own definition)."""
    M, N, K, r, s = 6, 16, 24, 8, 2.0
    W, A, B, X, dY = _rand_case(M, N, K, r, 11)
    w8 = Q.qlora_f8_quantize(W.to(DEV), Q.QLORA_F8_TILES, pow2=True)
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    x8 = Q.F8Matrix.empty(M, K, pow2=True)
    Q.qlora_f8_linear_fwd(w8, A.to(DEV), B.to(DEV), s * r, X.to(DEV), x8, U_save=U)
    dX, dA, dB = Q.qlora_f8_linear_bwd(w8, A.to(DEV), B.to(DEV), s * r, x8, U, dY.to(DEV),
                                       Q.QLORA_E4M3, check=True)
    xq = R.restore(*R.quantize(X, "rows", "e4m3", True), "rows", np.float64)
    wq = R.restore(*R.quantize(W, "tiles", "e4m3", True), "tiles", np.float64)
    dq = R.restore(*R.quantize(dY, "rows", "e4m3", True), "rows", np.float64)
    a, b, dy = _f(A), _f(B), _f(dY)

    def diff(f, v):
        g = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            h = 1e-4
            v[i] += h
            up = f()
            v[i] -= 2 * h
            g[i] = (up - f()) / (2 * h)
            v[i] += h
        return g
    # the loss is linear in each argument: differences are exact to rounding
    da = diff(lambda: float((dy * (s * (xq @ a.T) @ b.T)).sum()), a)
    db = diff(lambda: float((dy * (s * (_f(X) @ a.T) @ b.T)).sum()), b)
    x = xq.copy()
    dx = diff(lambda: float((dq * (x @ wq.T)).sum() + (dy * (s * (x @ a.T) @ b.T)).sum()), x)
    for got, want, tol in ((dA, da, 2.0 ** -14), (dB, db, 2.0 ** -14), (dX, dx, 2.0 ** -7)):
        assert np.abs(_f(got) - want).max() <= tol * np.abs(want).max()


@pytest.mark.parametrize("M", [300, 200])
def test_timed_and_counted(M):
    """With kernel timing on (event records between the launches) the results are the same.
    One launch quantises and multiplies by the adapter: 2 + 5 in all."""
    N, K, r = 256, 512, 16
    W, A, B, X, dY = (t.to(DEV) for t in _rand_case(M, N, K, r, 12))
    w8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES)
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)

    def step():
        x8 = Q.F8Matrix.empty(M, K)
        y = Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U, check=True)
        return [y, *Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY, check=True)]
    want, n0 = step(), Q.qlora_launch_count()
    Q.qlora_timing_begin([Q.QLORA_KERNEL_QUANTIZE, Q.QLORA_KERNEL_LORA_GEMM])
    got = step()
    t = Q.qlora_timing_end()
    assert Q.qlora_launch_count() - n0 == 7
    assert t[Q.QLORA_KERNEL_QUANTIZE][1] == 2 and t[Q.QLORA_KERNEL_LORA_GEMM][1] == 2
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K,r", [(1, 64, 72, 8), (3, 200, 1032, 24), (9, 136, 320, 72),
                                     (16, 128, 2048, 200), (37, 200, 328, 16),
                                     (130, 256, 704, 40), (520, 264, 448, 136)])
def test_workspace_holds_anything(M, N, K, r):
    """A workspace whose bytes past the status word are NaN gives the same results: nothing is
    read that the call did not write, padding included."""
    W, A, B, X, dY = (t.to(DEV) for t in _rand_case(M, N, K, r, 21))
    w8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES)
    q = Q.qlora_quantize(W) if K % 64 == 0 else None
    wf, wb = Q.qlora_f8_linear_workspace(M, N, K, r)
    need = (wf, wb, Q.qlora_linear_bwd_f8_workspace(M, N, K, r) if q else 0)

    def step(fill):
        ws = [torch.full((max(n, 256),), fill, dtype=torch.uint8, device=DEV) for n in need]
        for w in ws:
            w[:256] = 0
        x8 = Q.F8Matrix.empty(M, K)
        U = torch.empty((M, r), dtype=torch.float32, device=DEV)
        out = [Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U, workspace=ws[0], check=True),
               U, *Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY, workspace=ws[1], check=True)]
        if q:
            out += Q.qlora_linear_bwd_f8(q, A, B, r, 16.0, x8, U, dY, workspace=ws[2], check=True)
        return out
    for a, b in zip(step(0), step(0xff)):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("M,K,r", [(m, k, r) for m in (1, 5, 8, 9, 16) for k, r in (
    (8, 8), (136, 16), (1096, 40), (4096, 16), (11008, 64), (20000, 256))]
    + [(17, 8, 8), (33, 1096, 40), (100, 4096, 16), (250, 4096, 64), (256, 264, 256),
       (129, 2048, 136), (257, 128, 8), (40, 20000, 256), (300, 1096, 40), (520, 8, 8),
       (385, 11008, 64), (1000, 4096, 256), (2050, 520, 104)])
@pytest.mark.parametrize("fmt,pow2", [(Q.QLORA_E4M3, False), (Q.QLORA_E5M2, True)])
def test_codes_and_factor(M, K, r, fmt, pow2):
    """What the forward makes of X: the codes and scales of X that qlora_f8_quantize gives, U against fp64
    (sums of K terms: K e |x||A|^T), rows past the last token left as they were."""
    W, A, B, X, _ = _rand_case(M, 64, K, r, M + K + r)
    if K > 8:
        X[M - 1, 7], X[0, K - 1] = float("inf"), float("nan")
    X, A, B = X.to(DEV), A.to(DEV), B.to(DEV)
    w8 = Q.qlora_f8_quantize(W.to(DEV), Q.QLORA_F8_TILES)
    want = Q.qlora_f8_quantize(X, Q.QLORA_F8_ROWS, fmt, pow2)
    full = Q.F8Matrix.empty(M + 3, K, format=fmt, pow2=pow2)
    full.codes.fill_(77)
    x8 = Q.F8Matrix(M, K, Q.QLORA_F8_ROWS, fmt, pow2, full.codes[:M], torch.empty_like(want.scales))
    U = torch.full((M + 1, r), 5.0, device=DEV)
    Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U[:M], check=True)
    assert torch.equal(x8.codes, want.codes) and torch.equal(x8.scales, want.scales)
    assert (full.codes[M:] == 77).all() and (U[M:] == 5).all()
    x, a = _f(X), _f(A)
    bad = ~np.isfinite(x).all(axis=1)
    assert (~torch.isfinite(U[:M]).cpu().numpy())[bad].all()
    x = x[~bad]
    _within(U[:M].cpu()[torch.from_numpy(~bad)], x @ a.T, K * E * np.abs(x) @ np.abs(a).T, "U")


@pytest.mark.parametrize("M", [1, 12, 40, 200, 300])
def test_weight_written_just_before(M):
    """The product reads W while the launches ahead of it run: W, A and B written by the work
    right before the call, every time anew, give the results of calls that stand alone."""
    N, K, r = 1024, 2048, 16
    W, A, B, X, dY = (t.to(DEV) for t in _rand_case(M, N, K, r, 31))
    Ws, w8 = [W, (2 * W).flip(0), W.flip(1)], Q.F8Matrix.empty(N, K, Q.QLORA_F8_TILES)
    a, b, x8 = torch.empty_like(A), torch.empty_like(B), Q.F8Matrix.empty(M, K)
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)

    def step(i, wait):
        Q.qlora_f8_quantize(Ws[i], out=w8)
        a.copy_(A * (i + 1))
        b.copy_(B * (i + 1))
        if wait:
            torch.cuda.synchronize()
        out = [Q.qlora_f8_linear_fwd(w8, a, b, 16.0, X, x8, U_save=U)]
        Q.qlora_f8_quantize(Ws[(i + 1) % 3], out=w8)
        if wait:
            torch.cuda.synchronize()
        return out + list(Q.qlora_f8_linear_bwd(w8, a, b, 16.0, x8, U, dY))
    want = [step(i, True) for i in range(3)]
    torch.cuda.synchronize()
    for n in range(12):
        for x, y in zip(step(n % 3, False), want[n % 3]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("M", [3, 16, 50, 256, 300, 700])
def test_few_tokens_captured_and_without_dx(M):
    """Captured and replayed on new inputs; dA and dB without dX are those with it."""
    N, K, r = 264, 1096, 24
    W, A, B, X, dY = (t.to(DEV) for t in _rand_case(M, N, K, r, 41))
    w8 = Q.qlora_f8_quantize(W, Q.QLORA_F8_TILES)
    U = torch.empty((M, r), dtype=torch.float32, device=DEV)
    x8 = Q.F8Matrix.empty(M, K)

    def step():
        Y = Q.qlora_f8_linear_fwd(w8, A, B, 16.0, X, x8, U_save=U)
        return [Y, *Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    X.copy_(_rand((M, K), 42).to(DEV))
    dY.copy_(_rand((M, N), 43).to(DEV))
    graph.replay()
    want = step()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)
    none, dA, dB = Q.qlora_f8_linear_bwd(w8, A, B, 16.0, x8, U, dY, want_dx=False, check=True)
    assert none is None and torch.equal(dA, want[2]) and torch.equal(dB, want[3])

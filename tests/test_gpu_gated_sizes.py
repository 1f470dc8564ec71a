"""The gated block for few tokens where its adapters are large beside its weights (long reductions, rank 256, several token
groups), and the ends of the largest one."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import dev_bf16, host, log, require_gpu
from kv_cases import bits
from oracle import rows as oracle

pytestmark = pytest.mark.gpu

BF16, E24 = 2.0 ** -8, 2.0 ** -24
# M, in, out, r: adapter slices of 2048 rows take a quarter of the launch's workgroups, half, all, and more
CASES = [(64, 8192, 264, 128), (64, 8192, 264, 256), (33, 16384, 136, 256), (64, 16384, 520, 256), (17, 32768, 72, 200), (9, 65536, 40, 256)]


def _make(M, K, N, r):
    X = dev_bf16(bits(1, (M, K)))
    w = [Q.qlora_quantize_nf4(dev_bf16(bits(2 + i, (N, K), 0.02)), True) for i in range(2)]
    A = [dev_bf16(bits(4 + i, (K, r), 0.02)) for i in range(2)]
    B = [dev_bf16(bits(6 + i, (r, N), 0.02)) for i in range(2)]
    return X, w, A, B


def _check(X, w, A, B, scale, outs):
    """H, G, U and both X A against float64.  Tolerances: products exact in fp32, K of them added in some order (K 2^-24 of the sum
    of magnitudes, in slices of which it is far less), s T rounded to bf16 before its product with B, then one rounding; H:
    |act'| below 1.13, act within 2^-15."""
    H, G, U, Tg, Tu = outs
    K, r = A[0].shape
    f64 = lambda t: host(t.float()).astype(np.float64)
    x = f64(X)
    sums, tols = [], []
    for i, (got, gotT) in enumerate(((G, Tg), (U, Tu))):
        W, a, b = f64(Q.qlora_dequant(w[i])), f64(A[i]), f64(B[i])
        T, magT = x @ a, np.abs(x) @ np.abs(a)
        assert np.all(np.abs(f64(gotT) - T) <= BF16 * np.abs(T) + 1.01 * K * E24 * magT), i
        want = x @ W.T + scale * T @ b
        tol = 1.01 * (K + r + 16) * E24 * (np.abs(x) @ np.abs(W).T + scale * np.abs(T) @ np.abs(b))
        tol += 1.01 * scale * (BF16 * np.abs(T) + K * E24 * magT) @ np.abs(b)
        assert np.all(np.abs(f64(got) - want) <= 1.01 * BF16 * (np.abs(want) + tol) + tol), i
        sums.append(want)
        tols.append(tol)
    a = oracle.activation(sums[0], "silu")[0]
    want = a * sums[1]
    tol = 1.13 * tols[0] * (np.abs(sums[1]) + tols[1]) + np.abs(a) * tols[1] + 2.0 ** -15 * np.abs(want)
    assert np.all(np.abs(f64(H) - want) <= 1.01 * BF16 * (np.abs(want) + tol) + tol + 2.0 ** -126)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_large_adapters(case):
    require_gpu()
    log("gated few", case)
    X, w, A, B = _make(*case)
    outs = Q.qlora_gated_fwd(X, w[0], w[1], A[0], B[0], A[1], B[1], 0.25, "silu")
    _check(X, w, A, B, 0.25, outs)
    again = Q.qlora_gated_fwd(X, w[0], w[1], A[0], B[0], A[1], B[1], 0.25, "silu")
    assert all(torch.equal(p, q) for p, q in zip(again, outs))


def test_first_and_last_rows_of_the_largest_block():
    """260000 tokens of 8008 features: element by element, adapters' terms of the size of the products'."""
    require_gpu()
    M, tail = 260000, 300
    X, w, A, B = _make(tail, 64, 8008, 8)
    A = [a * 8 for a in A]
    big = torch.zeros(M, 64, dtype=torch.bfloat16, device="cuda")
    big[:tail], big[M - tail:] = X, X
    outs = Q.qlora_gated_fwd(big, w[0], w[1], A[0], B[0], A[1], B[1], 1.0, "silu")
    for rows in (slice(0, tail), slice(M - tail, M)):
        _check(X, w, A, B, 1.0, [t[rows] for t in outs])


def test_large_adapters_leave_room_for_the_weights():
    """The block in one launch takes no longer than its two products in launches of their own: half as much again is allowed here
    (it takes about 0.6 of them, and took 3.9 times as long where its adapters' workgroups left the weights a single range)."""
    require_gpu()
    X, w, A, B = _make(48, 22016, 8192, 256)
    ws = torch.empty(Q.qlora_gated_workspace(48, 22016, 8192, 256), dtype=torch.uint8, device="cuda")

    def block():
        Q.qlora_gated_fwd(X, w[0], w[1], A[0], B[0], A[1], B[1], 0.25, save=False, workspace=ws)

    def linears():
        for i in range(2):
            Q.qlora_linear_fwd(X, w[i], A[i], B[i], 0.25)

    def time(f):
        best = float("inf")
        for _ in range(8):
            t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            t[0].record()
            for _ in range(10):
                f()
            t[1].record()
            torch.cuda.synchronize()
            best = min(best, t[0].elapsed_time(t[1]))
        return best

    one, two = time(block), time(linears)
    log("gated few: block %.3f ms, two linear calls %.3f ms" % (one / 10, two / 10))
    assert one <= 1.5 * two

"""GPU parity of the residual RMS norm and its backward with the float64 oracle.

Tolerances, from the arithmetic: a result is rounded once to bf16 (half a step, 2^-8 of it).  Before that, sums over a
row of at most 32 products per thread, a tree of 6 steps in a wave and at most 15 additions across waves carry a relative
error of at most (32 + 6 + 15 + 4) 2^-24 of the sum of magnitudes, of which the root takes half; with the few single operations around them at
most 2^-18 of the magnitudes that are added.  Weight gradients are fp32 sums with such an error in each term and chains
of fewer than 2^9 additions: 2^-15 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_11_amd as Q
from helpers import dev_bf16, host, log, require_gpu
from kv_cases import bits
from oracle import rows as oracle

pytestmark = pytest.mark.gpu

BF16, FP32, SUM = 2.0 ** -8, 2.0 ** -18, 2.0 ** -15
# rows, dim: every number of threads and loads of a row, whole and partial
SHAPES = [(1, 8), (3, 64), (5, 504), (4, 512), (7, 520), (9, 1024), (5, 1032), (6, 2048), (3, 2056), (17, 4096), (2, 4104),
          (5, 5000), (3, 8192), (3, 8200), (2, 16384), (3, 16392), (2, 32768), (1200, 72), (2100, 256)]


def f64(t):
    return host(t.float()).astype(np.float64)


def _t(seed, shape, std=1.0):
    return dev_bf16(bits(seed, shape, std))


def _weight(seed, dim):
    return (1 + 0.3 * _t(seed, (dim,)).float()).bfloat16()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("res,weight", [(False, True), (True, True), (True, False)])
def test_forward(shape, res, weight):
    require_gpu()
    log("rms_norm", shape, res, weight)
    n, dim = shape
    x, r = _t(1, shape, 1.5), _t(2, shape, 3.0) if res else None
    w = _weight(3, dim) if weight else None
    y, h = Q.qlora_rms_norm(x, w, r, eps=1e-5)
    want, kept = oracle.rms_norm(f64(x), None if r is None else f64(r), None if w is None else f64(w), 1e-5)
    assert np.array_equal(f64(h), kept) and (h is x) == (r is None)
    assert np.all(np.abs(f64(y) - want) <= (BF16 + FP32) * np.abs(want))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dh,weight", [(False, True), (True, True), (True, False)])
def test_backward(shape, dh, weight):
    require_gpu()
    log("rms_norm_bwd", shape, dh, weight)
    n, dim = shape
    dy, h = _t(11, shape), _t(12, shape, 2.0)
    d = _t(13, shape) if dh else None
    w = _weight(14, dim) if weight else None
    dx, dw = Q.qlora_rms_norm_bwd(dy, h, w, d, eps=1e-5)
    F = lambda t: None if t is None else f64(t)
    want, want_w = oracle.rms_norm_bwd(f64(dy), f64(h), F(w), F(d), 1e-5)
    g = np.abs(f64(dy) if w is None else f64(dy) * f64(w))
    hh = np.abs(f64(h))
    r = 1 / np.sqrt((hh * hh).mean(-1, keepdims=True) + 1e-5)
    mag = r * (g + hh * r * r * (g * hh).mean(-1, keepdims=True)) + (0 if d is None else np.abs(f64(d)))
    assert np.all(np.abs(f64(dx) - want) <= BF16 * np.abs(want) + FP32 * mag)
    assert (dw is None) == (w is None)
    if dw is not None:
        assert np.all(np.abs(host(dw).astype(np.float64) - want_w) <= SUM * (np.abs(f64(dy)) * hh * r).sum(0))
        same, none = Q.qlora_rms_norm_bwd(dy, h, w, d, eps=1e-5, weight_grad=False)
        assert none is None and torch.equal(same, dx)


def test_difference():
    """The gradient against differences of the library's own forward, along a random direction: a step of 2^-6 of values
    near 1 moves the output by about 2^-6, whose rounding (2^-8 of values up to 4) averages out over 2^16 elements
    (2^-7 / 2^8 each way), and the curvature adds 2^-12: 2^-5 of the norm is far more than all of that."""
    require_gpu()
    shape = (64, 1024)
    x, v, dy = _t(21, shape), _t(22, shape), _t(23, shape)
    w = _weight(24, shape[1])
    dx, _ = Q.qlora_rms_norm_bwd(dy, x, w, eps=1e-5)
    step = 2.0 ** -6
    up, down = (x.double() + step * v.double()).bfloat16(), (x.double() - step * v.double()).bfloat16()
    y = [Q.qlora_rms_norm(t, w, eps=1e-5)[0].double() for t in (up, down)]
    moved = up.double() - down.double()
    a, b = ((y[0] - y[1]) * dy.double()).sum().item(), (moved * dx.double()).sum().item()
    scale = (moved.norm() * dx.double().norm()).item()
    assert abs(a - b) <= 2.0 ** -5 * scale


def test_strides_in_place_and_repeated():
    """Rows of wider buffers, outputs that are the inputs, broadcast rows, and the same bits every time."""
    require_gpu()
    n, dim = 37, 1048
    x, r = _t(1, (n, dim + 40)), _t(2, (n, dim + 8))
    w = _weight(3, dim)
    xv, rv = x[:, 16:16 + dim], r[:, :dim]
    y, h = Q.qlora_rms_norm(xv, w, rv)
    keep = x.clone(), r.clone()
    y2, h2 = Q.qlora_rms_norm(xv, w, rv, out=xv, sum_out=rv)
    assert y2 is xv and h2 is rv and torch.equal(y2, y) and torch.equal(h2, h)
    assert torch.equal(x[:, :16], keep[0][:, :16]) and torch.equal(x[:, 16 + dim:], keep[0][:, 16 + dim:])
    assert torch.equal(r[:, dim:], keep[1][:, dim:])
    one = _t(5, (1, dim)).expand(n, dim)
    y, h = Q.qlora_rms_norm(one, w, rv)
    assert torch.equal(y, Q.qlora_rms_norm(one.contiguous(), w, rv)[0])
    dy, dh = _t(6, (n, dim)), _t(7, (n, dim))
    a = Q.qlora_rms_norm_bwd(dy, h, w, dh)
    b = Q.qlora_rms_norm_bwd(dy, h, w, dh)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for dst in ("dy", "dh", "h"):
        t = {"dy": dy.clone(), "dh": dh.clone(), "h": h.clone()}
        dx, dw = Q.qlora_rms_norm_bwd(t["dy"], t["h"], w, t["dh"], dx=t[dst])
        assert dx is t[dst] and torch.equal(dx, a[0]) and torch.equal(dw, a[1])
    wide = torch.full((n, dim + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(Q.qlora_rms_norm_bwd(dy, h, w, one, dx=wide[:, 8:8 + dim])[0],
                       Q.qlora_rms_norm_bwd(dy, h, w, one.contiguous())[0])
    assert torch.all(wide[:, :8] == 7) and torch.all(wide[:, 8 + dim:] == 7)


def test_rows_past_32_bit_offsets():
    """Rows 2^31 + 40 elements apart: the last one lies 8.6 GB behind the first."""
    require_gpu()
    dim, stride = 1000, (1 << 31) + 40
    buf = torch.zeros(2 * stride + dim, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, dim), (stride, 1))
    small, r, dy = (_t(i, (3, dim)) for i in (1, 2, 3))
    w = _weight(4, dim)
    x.copy_(small)
    want, h = Q.qlora_rms_norm(small, w, r)
    assert torch.equal(Q.qlora_rms_norm(x, w, r)[0], want)
    Q.qlora_rms_norm(small, w, r, sum_out=x)
    assert torch.equal(x, h)
    dx, dw = Q.qlora_rms_norm_bwd(dy, h, w)
    got = Q.qlora_rms_norm_bwd(dy, x, w, dx=x)
    assert torch.equal(x, dx) and torch.equal(got[1], dw)
    assert buf[dim:stride].abs().max() == 0 and buf[stride + dim:2 * stride].abs().max() == 0


def test_no_rows_and_special_values():
    require_gpu()
    dim = 256
    e = torch.empty(0, dim, dtype=torch.bfloat16, device="cuda")
    w = _weight(1, dim)
    assert Q.qlora_rms_norm(e, w, e)[0].shape == (0, dim)
    dx, dw = Q.qlora_rms_norm_bwd(e, e, w)
    assert dx.shape == (0, dim) and torch.all(dw == 0)
    x = torch.zeros(4, dim, dtype=torch.bfloat16, device="cuda")
    x[1, 3] = float("inf")
    x[2, 3] = float("nan")
    x[3] = 2.0 ** -130   # (below the smallest normal number: its square is 0)
    y, _ = Q.qlora_rms_norm(x, w, eps=1e-6)
    assert torch.all(y[0] == 0) and y[1].isnan().sum() == 1 and y[2].isnan().all() and torch.all(y[3].abs() < 1e-30)
    dx, dw = Q.qlora_rms_norm_bwd(torch.ones_like(x)[:1], x[:1], w, eps=1e-6)
    assert torch.equal(dx, (w.float() / np.sqrt(1e-6)).bfloat16()[None]) or \
        torch.all((dx.float() - w.float() * 1e3).abs() <= (BF16 + FP32) * w.float().abs() * 1e3)
    assert torch.all(dw == 0)


def test_captured_and_other_streams():
    require_gpu()
    n, dim = 300, 2048
    x, r, dy, dh = (_t(i, (n, dim)) for i in range(4))
    w = _weight(9, dim)
    ws = torch.empty(Q.qlora_rms_norm_bwd_workspace(n, dim), dtype=torch.uint8, device="cuda")

    def run():
        y, h = Q.qlora_rms_norm(x, w, r)
        return (y, h, *Q.qlora_rms_norm_bwd(dy, h, w, dh, workspace=ws))

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for k in (1, 2, 3):
        for i, t in enumerate((x, r, dy, dh)):
            t.copy_(_t(10 * k + i, (n, dim)))
        eager = [t.clone() for t in run()]
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h = Q.qlora_rms_norm(x, w, r, stream=side)
    got = Q.qlora_rms_norm_bwd(dy, h, w, dh, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, h, *got), eager))


def test_binding_refusals():
    require_gpu()
    x = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros(5, 68, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x.cpu(), x[0], x[:, ::2], odd, odd[:, :64], odd[:, 4:], x[None]):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_rms_norm(bad, None)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_rms_norm_bwd(bad, x, None)
        with pytest.raises(Q.QLoRAError):
            Q.qlora_rms_norm_bwd(x, bad, None)
    for bad in (x[:4], x.cpu(), x.float(), torch.zeros(5, 72, dtype=torch.bfloat16, device="cuda")):
        for kw in ({"residual": bad}, {"out": bad}, {"residual": x, "sum_out": bad}):
            with pytest.raises(Q.QLoRAError):
                Q.qlora_rms_norm(x, w, **kw)
        for kw in ({"dh": bad}, {"dx": bad}):
            with pytest.raises(Q.QLoRAError):
                Q.qlora_rms_norm_bwd(x, x, w, **kw)
    for bad in (w.float(), w[:32], w.cpu(), w.expand(2, 64)):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_rms_norm(x, bad)
    same = x.clone()
    for kw in ({"sum_out": x}, {"eps": -1.0}, {"eps": float("nan")}, {"residual": x, "out": same, "sum_out": same}):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_rms_norm(x, w, **kw)
    for kw in ({"dweight": torch.zeros(32, device="cuda")}, {"dweight": torch.zeros(64, device="cuda"), "weight_grad": False},
               {"workspace": torch.empty(64, dtype=torch.uint8, device="cuda")}):
        with pytest.raises(Q.QLoRAError):
            Q.qlora_rms_norm_bwd(x, x, w, **kw)
